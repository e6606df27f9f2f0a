"""Attention over 4-bit caches on the GPU, through every entry point that reads a cache, against
the fp64 reference and bounds of fp4_cases.py."""
import numpy as np
import pytest
import torch

import fp4_cases
import oracle

import paged_decode_attention_reshape_gb300 as pa

pytestmark = pytest.mark.gpu

PARTS = [-1, 64, 0, -2, -8, pa.PA_PARTITION_BALANCED]
LENS = [0, 1, 17, 100, 700, 1100]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    pa.lib()
    torch.cuda.set_device(0)


def _decode(c, g, P=0, ws=True, **kw):
    g.out.fill_(float("nan"))
    pa.pa_decode_opt(g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, c.Hkv,
                     k_scale=g.k_scale, v_scale=g.v_scale, scale_stride=g.stride, alibi_slopes=g.alibi,
                     partition_size=P, workspace=g.ws if ws else None, device_error=g.err, **kw)
    return pa.pa_check_device_error(g.err)


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 64), (32, 8, 64), (32, 8, 128), (64, 8, 128), (6, 2, 128), (16, 1, 256),
                                      (9, 3, 256), (40, 2, 64)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_decode(Hq, Hkv, D, dt):
    c = fp4_cases.make(len(LENS), Hq, Hkv, D, LENS, dt, seed=Hq + D, k_scale=0.31, v_scale=2.5)
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    for P in PARTS:
        assert _decode(c, g, P) == (0, 0)
        fp4_cases.check(g.out, ref, tol, "partition %d" % P)
    assert _decode(c, g, 64, ws=False) == (0, 0)
    fp4_cases.check(g.out, ref, tol, "library workspace")


def test_decode_per_head_scales_interleaved_pages_strided_rows():
    Hq, Hkv, D = 24, 4, 128
    heads = np.array([0.05, 0.37, 1.0, 3.0], np.float32)
    c = fp4_cases.make(len(LENS), Hq, Hkv, D, LENS, seed=5, k_scale=heads, v_scale=heads[::-1].copy(), interleaved=True)
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    wide = torch.full((c.S, 3, Hq, D), float("nan"), dtype=c.dtype, device="cuda")   # q and out inside wider rows
    wide[:, 1] = g.q
    out = torch.full((c.S, 2, Hq, D), float("nan"), dtype=c.dtype, device="cuda")
    g.q, g.out = wide[:, 1], out[:, 0]
    for P in (-1, 128, pa.PA_PARTITION_BALANCED):
        assert _decode(c, g, P) == (0, 0)
        fp4_cases.check(g.out, ref, tol, "partition %d" % P)
    assert bool(out[:, 1].isnan().all())


@pytest.mark.parametrize("sigma", [1e-3, 30.0, 400.0])
def test_decode_magnitudes(sigma):
    """Values near the scales' lower end, and logits of thousands (one token takes all)."""
    c = fp4_cases.make(3, 8, 2, 128, [1, 40, 333], torch.bfloat16, seed=7, sigma=sigma)
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    for P in (-1, 64):
        assert _decode(c, g, P) == (0, 0)
        fp4_cases.check(g.out, ref, tol, "sigma %g partition %d" % (sigma, P))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_alibi(D):
    slopes = 2.0 ** -np.arange(1, 9)
    c = fp4_cases.make(len(LENS), 8, 2, D, LENS, seed=D, alibi=slopes)
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    for P in (-1, 64, 0):
        assert _decode(c, g, P) == (0, 0)
        fp4_cases.check(g.out, ref, tol, "partition %d" % P)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (32, 8, 128), (8, 4, 256)])
@pytest.mark.parametrize("alibi", [False, True])
def test_varlen(Hq, Hkv, D, alibi):
    """Several query tokens per sequence, long chunks too (they run in columns of 8)."""
    lens, nq = [5, 1, 210, 64, 300], [5, 1, 3, 0, 40]
    slopes = 2.0 ** (-8 * np.arange(1, Hq + 1) / Hq) if alibi else None
    c = fp4_cases.make(5, Hq, Hkv, D, lens, torch.float16, seed=D + 1, nq=nq, alibi=slopes, k_scale=0.5)
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    for P in (0, -1, 64, -2):
        g.out.fill_(float("nan"))
        pa.pa_attention_varlen(g.out, g.q, g.k_cache, g.v_cache, g.starts, g.block_table, g.seq_lens, c.scale, Hkv,
                               max(nq), k_scale=g.k_scale, v_scale=g.v_scale, alibi_slopes=g.alibi,
                               partition_size=P, device_error=g.err)
        assert pa.pa_check_device_error(g.err) == (0, 0)
        fp4_cases.check(g.out, ref, tol, "partition %d" % P)


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_step_equals_write_then_decode(rows, D):
    """pa_decode_step: the newest rows quantised and written, then attended to; the same bytes and
    outputs as the two calls, which the oracle checks."""
    Hq, Hkv = 16, 4
    lens = [rows, 40, 130, 17 + rows]
    c = fp4_cases.make(4, Hq, Hkv, D, lens, seed=3 + rows, k_scale=0.4, v_scale=0.6)
    T = 4 * rows
    rng = np.random.RandomState(8)
    new = [torch.from_numpy(rng.randn(T, Hkv, D).astype(np.float32)).to(torch.bfloat16) for _ in range(2)]
    slots = []
    for s, L in enumerate(lens):
        pos = np.arange(L - rows, L)
        slots += list(c.table[s][pos // 16].astype(np.int64) * 16 + pos % 16)
        for vals, x, sc in ((c.K, new[0], 0.4), (c.V, new[1], 0.6)):
            code, sg = oracle.fp4_quantize(x[s * rows:(s + 1) * rows].float().numpy(), sc)
            vals[s][L - rows:] = oracle.fp4_values(code, sg, sc)
    ref, tol, _ = fp4_cases.reference(c)
    slots = torch.tensor(slots, device="cuda")
    starts = None if rows == 1 else torch.arange(5, dtype=torch.int32, device="cuda") * rows
    a, b = fp4_cases.to_gpu(c), fp4_cases.to_gpu(c)
    kw = dict(k_scale=a.k_scale, v_scale=a.v_scale)
    for P in (0, 64, -2):
        pa.pa_decode_step(a.out, a.q, new[0].cuda(), new[1].cuda(), a.k_cache, a.v_cache, slots, a.block_table,
                          a.seq_lens, c.scale, Hkv, new_rows_start=starts, partition_size=P, device_error=a.err, **kw)
        assert pa.pa_check_device_error(a.err) == (0, 0)
        fp4_cases.check(a.out, ref, tol, "step, partition %d" % P)
        pa.pa_reshape_and_cache(new[0].cuda(), new[1].cuda(), b.k_cache, b.v_cache, slots, pa.PA_KV_FP4_E2M1, **kw)
        assert _decode(c, b, P) == (0, 0)
        assert torch.equal(a.out, b.out)
        assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.v_cache, b.v_cache)


def test_other_entry_points_agree():
    c = fp4_cases.make(3, 8, 2, 128, [900, 33, 500], seed=1)
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    args = (g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, c.Hkv)
    for name, call in (("pa_decode", lambda: pa.pa_decode(*args)),
                       ("pa_decode_ex", lambda: pa.pa_decode_ex(*args, g.k_scale, g.v_scale, 128, g.ws, g.err)),
                       ("pa_decode_noalloc", lambda: pa.pa_decode_noalloc(*args, partition_size=64))):
        g.out.fill_(float("nan"))
        call()
        fp4_cases.check(g.out, ref, tol, name)


def test_long_context():
    """One sequence over more pages than a warp's table registers hold, split and unsplit."""
    c = fp4_cases.make(1, 4, 1, 64, [9000], torch.float16, seed=4)
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    for P in (-1, 0, 1024, 16):
        assert _decode(c, g, P) == (0, 0)
        fp4_cases.check(g.out, ref, tol, "partition %d" % P)


def test_nan_group_reaches_its_head_only():
    c = fp4_cases.make(2, 4, 2, 128, [30, 20], seed=6)
    place = oracle.fp4_place(128)
    c.pool[1][c.table[0, 1], 1, place[3, 64 + 2]] = 0x7F       # V scale of token 19, head 1, elements 32 .. 47
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    assert _decode(c, g, -1) == (0, 0)
    got = g.out.double().cpu().numpy()
    nan = np.zeros(got.shape, bool)
    nan[0, 2:, 32:48] = True
    assert np.array_equal(np.isnan(got), nan)
    assert (np.abs(got - ref) <= tol)[~nan].all()


def test_bad_table_entry_and_length_write_nothing():
    c = fp4_cases.make(3, 8, 2, 64, [100, 200, 50], seed=2)
    ref, tol, _ = fp4_cases.reference(c)
    for P in (-1, 64, -2):
        g = fp4_cases.to_gpu(c)
        g.block_table[0, 3] = c.NB
        g.seq_lens[2] = c.width * 16 + 1
        rc, bits = _decode(c, g, P)
        assert rc == -6 and bits == pa.PA_DEVERR_BLOCK_RANGE | pa.PA_DEVERR_SEQLEN_RANGE
        assert bool(g.out[0].isnan().all()) and bool(g.out[2].isnan().all())
        fp4_cases.check(g.out[1], ref[1], tol[1], "the sequence without a fault")


def test_other_stream_and_graph():
    c = fp4_cases.make(4, 32, 8, 128, [700, 3, 0, 250], seed=9)
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    args = (g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, c.Hkv)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        g.out.fill_(float("nan"))
        pa.pa_decode_opt(*args, partition_size=64, workspace=g.ws)
    stream.synchronize()
    fp4_cases.check(g.out, ref, tol, "another stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pa.pa_decode_opt(*args, partition_size=64, workspace=g.ws)
    for _ in range(2):
        g.out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        fp4_cases.check(g.out, ref, tol, "replay")


# ------------------------------------------------ the split over warps (many sequences and heads)

def _many(Hq, Hkv, D, dt, S, seed, **kw):
    rng = np.random.RandomState(seed)
    lens = (rng.rand(S) ** 3 * 900).astype(int)      # most short, some long
    lens[:8] = [0, 1, 16, 17, 63, 64, 65, 1500]
    lens[-2:] = [700, 0]
    return fp4_cases.make(S, Hq, Hkv, D, lens.tolist(), dt, seed=seed, **kw)


@pytest.mark.parametrize("Hq,Hkv,D,S,dt", [(16, 8, 64, 60, torch.bfloat16), (8, 8, 128, 50, torch.float16),
                                           (20, 10, 128, 40, torch.bfloat16), (36, 4, 64, 50, torch.bfloat16),
                                           (12, 6, 256, 60, torch.float16)])
def test_split_over_warps(Hq, Hkv, D, S, dt):
    c = _many(Hq, Hkv, D, dt, S, seed=D + S, k_scale=0.7, v_scale=1.3, interleaved=D == 128)
    B = pa.PA_PARTITION_BALANCED
    assert pa.pa_decode_plan(S, Hq, Hkv, D, c.width, pa.PA_FP4_E2M1, partition_size=B)[1] % 4 == 0
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    first = None
    for P, ws in ((B, True), (B, False), (B, True)):
        assert _decode(c, g, P, ws=ws) == (0, 0)
        fp4_cases.check(g.out, ref, tol, "partition %d" % P)
        first = g.out.clone() if first is None else first
        assert torch.equal(first, g.out)              # the parts merge in order, whoever merges them
    size = pa.pa_decode_workspace_size(S, Hq, Hkv, D, c.width, pa.PA_PARTITION_BALANCED)
    g.ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    assert _decode(c, g, B) == (0, 0) and torch.equal(first, g.out)
    # the size also serves the same shape's other plans
    slopes = torch.full((Hq,), 0.01, device="cuda")
    g.ws.zero_()
    pa.pa_decode_opt(g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, Hkv, alibi_slopes=slopes,
                     workspace=g.ws, device_error=g.err)
    assert pa.pa_check_device_error(g.err) == (0, 0)


def test_split_over_warps_is_the_plan_of_many_units():
    c = _many(8, 8, 64, torch.bfloat16, 210, seed=8)
    assert pa.pa_decode_plan(210, 8, 8, 64, c.width, pa.PA_FP4_E2M1)[0] == pa.PA_PARTITION_BALANCED
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    assert _decode(c, g, 0, ws=False) == (0, 0)
    fp4_cases.check(g.out, ref, tol)
    first = g.out.clone()
    assert _decode(c, g, pa.PA_PARTITION_BALANCED) == (0, 0)
    assert torch.equal(first, g.out)


def test_split_over_warps_faults_and_recovery():
    c = _many(16, 8, 64, torch.bfloat16, 60, seed=77)
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    good = (g.block_table.clone(), g.seq_lens.clone())
    long = int(np.argmax(c.lens))
    g.block_table[long, 40] = -5                       # inside a sequence that several warps share
    g.block_table[4, 0] = c.NB
    g.seq_lens[20] = -1
    for _ in range(2):
        rc, bits = _decode(c, g, pa.PA_PARTITION_BALANCED)
        assert rc == -6 and bits == pa.PA_DEVERR_BLOCK_RANGE | pa.PA_DEVERR_SEQLEN_RANGE
        bad = [long, 4, 20]
        assert bool(g.out[bad].isnan().all())
        keep = [s for s in range(c.S) if s not in bad]
        fp4_cases.check(g.out[keep], ref[keep], tol[keep], "sequences without a fault")
    g.block_table, g.seq_lens = good
    assert _decode(c, g, pa.PA_PARTITION_BALANCED) == (0, 0)                  # the counters are back at zero
    fp4_cases.check(g.out, ref, tol, "after the faults")


def test_split_over_warps_empty_and_equal_batches():
    for lens in ([0] * 60, [1] * 60, [64] * 60, [5] + [0] * 58 + [3]):
        c = fp4_cases.make(60, 8, 8, 64, lens, torch.bfloat16, seed=3)
        ref, tol, _ = fp4_cases.reference(c)
        g = fp4_cases.to_gpu(c)
        assert _decode(c, g, pa.PA_PARTITION_BALANCED) == (0, 0)
        fp4_cases.check(g.out, ref, tol, str(lens[:3]))


def test_split_over_warps_in_two_graphs_of_one_workspace():
    """Two captured calls of different shapes on the library's workspace, replayed in turn."""
    cases = [_many(16, 8, 64, torch.bfloat16, 60, seed=1), _many(8, 8, 128, torch.bfloat16, 45, seed=2)]
    stream, graphs, on = torch.cuda.Stream(), [], []
    for c in cases:
        g = fp4_cases.to_gpu(c)
        assert _decode(c, g, pa.PA_PARTITION_BALANCED, ws=False) == (0, 0)
        on.append((c, g, *fp4_cases.reference(c)[:2]))
    for c, g, _, _ in on:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            pa.pa_decode_opt(g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, c.Hkv,
                             k_scale=g.k_scale, v_scale=g.v_scale, partition_size=pa.PA_PARTITION_BALANCED)
    for i in (0, 1, 1, 0):
        c, g, ref, tol = on[i]
        g.out.fill_(float("nan"))
        torch.cuda.synchronize()
        graphs[i].replay()
        torch.cuda.synchronize()
        fp4_cases.check(g.out, ref, tol, "graph %d" % i)


def test_more_sequences_than_the_balanced_split_takes():
    c = fp4_cases.make(520, 2, 1, 64, [i % 40 for i in range(520)], torch.bfloat16, seed=4)
    ref, tol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    assert _decode(c, g, 0) == (0, 0)
    fp4_cases.check(g.out, ref, tol, "520 sequences")


# ------------------------------------------------------------------------- far offsets

def _far_case(c, kc, vc, base):
    """Case c's pages moved to blocks base .. of larger caches."""
    kc[base:base + c.NB] = torch.from_numpy(c.pool[0]).cuda()
    vc[base:base + c.NB] = torch.from_numpy(c.pool[1]).cuda()
    return torch.from_numpy(np.where(c.table >= 0, c.table + base, -1).astype(np.int32)).cuda()


def test_caches_past_4_gib():
    """Pages, rows read back, rows written and rows moved at byte offsets above 2^32."""
    D, Hkv = 128, 8
    c = fp4_cases.make(3, 16, Hkv, D, [300, 40, 1], seed=12)
    base = (1 << 32) // (Hkv * 9 * D) + 1000
    NB = base + c.NB
    kc = torch.empty(NB, Hkv, 9 * D, dtype=torch.uint8, device="cuda")
    vc = torch.empty_like(kc)
    g = fp4_cases.to_gpu(c)
    g.block_table = _far_case(c, kc, vc, base)
    g.k_cache, g.v_cache = kc, vc
    ref, tol, _ = fp4_cases.reference(c)
    for P in (-1, 64):
        assert _decode(c, g, P) == (0, 0)
        fp4_cases.check(g.out, ref, tol, "partition %d" % P)
    slots = (g.block_table[0, :3].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()
    key = torch.zeros(48, Hkv, D, device="cuda")
    value = torch.zeros_like(key)
    pa.pa_gather_cache(key, value, kc, vc, slots)
    assert np.array_equal(key.double().cpu().numpy(), c.K[0][:48])
    assert np.array_equal(value.double().cpu().numpy(), c.V[0][:48])
    pa.pa_reshape_and_cache(value, key, kc, vc, slots, pa.PA_KV_FP4_E2M1)      # swapped: values of the format stay
    pa.pa_gather_cache(key, value, kc, vc, slots)
    assert np.abs(key.double().cpu().numpy() - c.V[0][:48]).max() <= 0.5 * np.abs(c.V[0][:48]).max()
    w = torch.arange(c.width * 16, device="cuda", dtype=torch.float32).expand(3, Hkv, -1).contiguous()
    kept = torch.zeros(3, Hkv, 100, dtype=torch.int32, device="cuda")
    nl, nw = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros_like(w)
    pa.pa_evict(kc, vc, g.block_table, g.seq_lens, w, 100, 0, kept, nl, nw)
    assert kept[0, 0, 0] == 200 and nl.tolist() == [100, 40, 1]
    pa.pa_gather_cache(key, value, kc, vc, slots)
    assert np.array_equal(key.double().cpu().numpy(), c.K[0][200:248])
    assert np.array_equal(value.double().cpu().numpy(), c.V[0][200:248])


def test_block_stride_past_2_gib():
    """Strides that a 32-bit number does not hold (the write's and the read back's other variant)."""
    D, far = 64, (1 << 31) + 4096
    c = fp4_cases.make(1, 2, 1, D, [30], seed=13)
    raw = torch.empty(far + c.NB * 9 * D, dtype=torch.uint8, device="cuda")
    kc = raw.as_strided((2, 1, 9 * D), (far, 9 * D, 1))
    rows = torch.from_numpy(np.random.RandomState(1).randn(32, 1, D).astype(np.float32)).cuda()
    slots = torch.arange(32, device="cuda")
    vc = torch.zeros(2, 1, 9 * D, dtype=torch.uint8, device="cuda")
    pa.pa_reshape_and_cache(rows, rows, kc, vc, slots, pa.PA_KV_FP4_E2M1)
    assert torch.equal(kc[0], vc[0]) and torch.equal(kc[1], vc[1])
    a, b = torch.zeros_like(rows), torch.zeros_like(rows)
    pa.pa_gather_cache(a, b, kc, vc, slots)
    assert torch.equal(a, b) and bool(a.any())
    out, ref = torch.zeros(1, 2, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 2, D, dtype=torch.bfloat16, device="cuda")
    bt, sl = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), torch.tensor([30], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 2, D, device="cuda").to(torch.bfloat16)
    pa.pa_decode(out, q, kc, kc, bt, sl, 0.1, 1)
    pa.pa_decode(ref, q, vc, vc, bt, sl, 0.1, 1)
    assert torch.equal(out, ref)
