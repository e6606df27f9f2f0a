"""pa_decode_accumulate on the GPU: the decode's outputs as pa_decode_opt writes them, and the
accumulated attention weights against fp64, over every cache type.

Bound of an accumulated weight: the array's entry w plus sum_h p_h, with p_h = 2^(s_h - lse_h).  A
logit is off by at most e (fp4_cases.py's: (D / 16 + 4) 2^-22 B), and so is the log of the softmax
sum, whose fp32 sum over L tokens adds (L / 16 + 32) 2^-24; the difference of the two is rounded
once, 2^-24 of a number below 1.45 B + log2 L + 8; 2^x is good to 2^-22; G additions and the one to
w round to 2^-24 each."""
import math

import numpy as np
import pytest
import torch

import fp4_cases
from gpu_cases import make_case, to_gpu

import paged_decode_attention_reshape_gb300 as pa

pytestmark = pytest.mark.gpu

LENS = [0, 1, 17, 100, 700, 1100]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    pa.lib()
    torch.cuda.set_device(0)


def expected(c, K, before):
    """fp64 weights after one call on `before` [S, Hkv, W], and their bounds."""
    q = c.q.double().numpy()
    want, tol = before.astype(np.float64), np.zeros(before.shape)
    G = c.Hq // c.Hkv
    for s, L in enumerate(c.lens):
        for h in range(c.Hq if L else 0):
            k = K[s][:, h // G]
            x, B = k @ q[s, h] * c.scale, np.abs(k) @ np.abs(q[s, h]) * c.scale
            if c.alibi is not None:
                bias = np.float64(c.alibi[h]) * (np.arange(L) - (L - 1))
                x, B = x + bias, B + np.abs(bias)
            p = np.exp(x - x.max())
            p /= p.sum()
            B = B.max()
            e = (c.D / 16 + 4) * 2.0 ** -22 * B
            want[s, h // G, :L] += p
            tol[s, h // G, :L] += p * (2 * e + (L / 16 + 32) * 2.0 ** -24 + (1.45 * B + math.log2(L) + 8) * 2.0 ** -24
                                       + 2.0 ** -22 + G * 2.0 ** -24) + 2.0 ** -120
    tol += 2.0 ** -24 * np.abs(want)
    return want, tol


def _case(kind, Hq, Hkv, D, alibi=None):
    """(case, GPU tensors, K values, K scale, V scale)."""
    if kind == "fp4":
        c = fp4_cases.make(len(LENS), Hq, Hkv, D, LENS, seed=D + Hq, k_scale=0.4, v_scale=0.6, alibi=alibi)
        return c, fp4_cases.to_gpu(c), c.K
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.bfloat16}[kind]
    c = make_case(len(LENS), Hq, Hkv, D, LENS, dtype=dt, fp8=kind == "e4m3", seed=D + Hq, alibi=alibi,
                  k_scale=0.05 if kind == "e4m3" else 1.0, v_scale=0.07 if kind == "e4m3" else 1.0)
    return c, to_gpu(c), c.Kval


def _args(c, g):
    return (g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, c.Hkv)


def _kw(kind, g):
    return dict(k_scale=g.k_scale, v_scale=g.v_scale) if kind in ("fp4", "e4m3") else {}


SHAPES = [("bf16", 32, 8, 64), ("bf16", 24, 8, 128), ("f16", 6, 6, 256), ("e4m3", 64, 8, 128), ("e4m3", 8, 4, 256),
          ("f32", 8, 2, 64), ("f32", 12, 1, 128), ("fp4", 32, 8, 128), ("fp4", 10, 5, 64), ("fp4", 20, 1, 256)]


@pytest.mark.parametrize("kind,Hq,Hkv,D", SHAPES, ids=["%s-%d-%d-%d" % s for s in SHAPES])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "alibi"])
def test_weights_and_outputs(kind, Hq, Hkv, D, biased):
    c, g, K = _case(kind, Hq, Hkv, D, 2.0 ** (-8 * np.arange(1, Hq + 1) / Hq) if biased else None)
    W = g.block_table.shape[1] * 16 + 3
    rng = np.random.RandomState(1)
    before = np.exp(rng.randn(c.S, Hkv, W)).astype(np.float32)
    want, tol = expected(c, K, before)
    alibi = None if c.alibi is None else torch.from_numpy(np.asarray(c.alibi, np.float32)).cuda()
    for P in (-1, 64, 0, pa.PA_PARTITION_BALANCED):
        outs = []
        for ws in (None, torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")):
            wide = torch.full((c.S, 2, Hkv, W), float("nan"), device="cuda")      # a strided array
            weights = wide[:, 1]
            weights.copy_(torch.from_numpy(before))
            g.out.fill_(float("nan"))
            pa.pa_decode_accumulate(*_args(c, g), weights, alibi_slopes=alibi, partition_size=P, workspace=ws,
                                    device_error=g.err, **_kw(kind, g))
            assert pa.pa_check_device_error(g.err) == (0, 0)
            got = weights.double().cpu().numpy()
            bad = ~(np.abs(got - want) <= tol)
            assert not bad.any(), (P, np.argwhere(bad)[:4], np.abs(got - want)[bad][:4], tol[bad][:4])
            for s, L in enumerate(LENS):
                assert np.array_equal(got[s, :, L:], before[s, :, L:])
            assert bool(wide[:, 0].isnan().all())
            outs.append(g.out.clone())
        assert torch.equal(outs[0], outs[1])
        g.out.fill_(float("nan"))
        pa.pa_decode_opt(*_args(c, g), alibi_slopes=alibi, partition_size=P, device_error=g.err, **_kw(kind, g))
        assert torch.allclose(outs[0].float(), g.out.float(), rtol=2.0 ** -7, atol=1e-5)


def test_repeated_calls_add_up():
    c, g, K = _case("bf16", 32, 8, 64)
    W = g.block_table.shape[1] * 16
    weights = torch.zeros(c.S, c.Hkv, W, device="cuda")
    for _ in range(5):
        pa.pa_decode_accumulate(*_args(c, g), weights)
    want, tol = expected(c, K, np.zeros(weights.shape, np.float32))
    got = weights.double().cpu().numpy()
    assert (np.abs(got - 5 * want) <= 5 * tol + 5 * 2.0 ** -24 * np.abs(5 * want)).all()
    total = got.sum(-1)
    for s, L in enumerate(LENS):     # every call adds one per query head
        assert np.allclose(total[s], 5 * 4 if L else 0, atol=1e-3)


@pytest.mark.parametrize("kind", ["bf16", "fp4", "f32"])
def test_faults_add_nothing(kind):
    c, g, K = _case(kind, 8, 2, 64)
    W = g.block_table.shape[1] * 16
    want, tol = expected(c, K, np.zeros((c.S, 2, W), np.float32))
    g.block_table[4, 5] = -3
    g.seq_lens[3] = W + 1
    g.seq_lens[1] = -1
    for P in (-1, 64, 0, pa.PA_PARTITION_BALANCED):
        weights = torch.zeros(c.S, 2, W, device="cuda")
        pa.pa_decode_accumulate(*_args(c, g), weights, partition_size=P, device_error=g.err, **_kw(kind, g))
        assert pa.pa_check_device_error(g.err) == (-6, pa.PA_DEVERR_BLOCK_RANGE | pa.PA_DEVERR_SEQLEN_RANGE)
        got = weights.double().cpu().numpy()
        assert not got[[1, 3, 4]].any()
        assert (np.abs(got - want) <= tol)[[0, 2, 5]].all()


def test_timed_out_wait_adds_nothing():
    c, g, _ = _case("bf16", 8, 2, 64)
    weights = torch.zeros(c.S, 2, g.block_table.shape[1] * 16, device="cuda")
    for P in (-1, 64):
        pa.pa_decode_accumulate(*_args(c, g), weights, partition_size=P, device_error=g.err, first_wait_limit=-1)
        assert pa.pa_check_device_error(g.err) == (-8, pa.PA_DEVERR_WAIT_TIMEOUT)
        assert not bool(weights.any())


def test_captured_after_a_first_call():
    c, g, K = _case("fp4", 32, 8, 128)
    W = g.block_table.shape[1] * 16
    weights = torch.zeros(c.S, c.Hkv, W, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        pa.pa_decode_accumulate(*_args(c, g), weights, **_kw("fp4", g))
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pa.pa_decode_accumulate(*_args(c, g), weights, **_kw("fp4", g))
    weights.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    want, tol = expected(c, K, np.zeros(weights.shape, np.float32))
    assert (np.abs(weights.double().cpu().numpy() - want) <= tol).all()


def test_many_sequences_over_a_4_bit_cache():
    """The decode's split over warps (parts of a sequence merged by the last warp to finish)."""
    rng = np.random.RandomState(5)
    lens = (rng.rand(60) ** 3 * 900).astype(int)
    lens[:5] = [0, 1, 64, 65, 1300]
    c = fp4_cases.make(60, 16, 8, 128, lens.tolist(), torch.bfloat16, seed=9)
    B = pa.PA_PARTITION_BALANCED
    ref, otol, _ = fp4_cases.reference(c)
    g = fp4_cases.to_gpu(c)
    W = c.width * 16
    before = np.exp(rng.randn(60, 8, W)).astype(np.float32)
    want, tol = expected(c, c.K, before)
    size = pa.pa_decode_accumulate_workspace_size(60, 16, 8, 128, c.width, B)
    for ws in (None, torch.zeros(size, dtype=torch.uint8, device="cuda")):
        weights = torch.from_numpy(before).cuda()
        pa.pa_decode_accumulate(*_args(c, g), weights, partition_size=B, workspace=ws, device_error=g.err)
        assert pa.pa_check_device_error(g.err) == (0, 0)
        fp4_cases.check(g.out, ref, otol, "outputs")
        assert (np.abs(weights.double().cpu().numpy() - want) <= tol).all()
    g.block_table[4, 50] = -1
    g.block_table[2, 0] = -1
    weights = torch.zeros(60, 8, W, device="cuda")
    pa.pa_decode_accumulate(*_args(c, g), weights, partition_size=B, device_error=g.err)
    assert pa.pa_check_device_error(g.err) == (-6, pa.PA_DEVERR_BLOCK_RANGE)
    got = weights.double().cpu().numpy()
    assert not got[[2, 4]].any() and got[3].any()


def test_one_column_tables_and_tokens():
    """The shortest call: one sequence of one token, whose weight is 1 for every query head."""
    for kind in ("fp4", "bf16"):
        c = fp4_cases.make(1, 4, 2, 64, [1], torch.bfloat16, seed=1) if kind == "fp4" else make_case(
            1, 4, 2, 64, [1], seed=1)
        g = fp4_cases.to_gpu(c) if kind == "fp4" else to_gpu(c)
        weights = torch.full((1, 2, g.block_table.shape[1] * 16), 0.25, device="cuda")
        pa.pa_decode_accumulate(*_args(c, g), weights, device_error=g.err)
        assert pa.pa_check_device_error(g.err) == (0, 0)
        assert torch.allclose(weights[:, :, 0], torch.full((1, 2), 2.25, device="cuda"), atol=1e-6)
        assert bool((weights[:, :, 1:] == 0.25).all())
