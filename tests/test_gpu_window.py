"""pa_decode_window and pa_attention_window on the GPU against fp64 (window_cases.py): every cache type,
head size, split and kernel, with windows and first tokens that end anywhere in a page, and everything that
no query sees poisoned."""
import numpy as np
import pytest
import torch

import paged_decode_attention_reshape_gb300 as pa
import window_cases as wc

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
BAL = pa.PA_PARTITION_BALANCED

# (cache, dtype, head size, query heads per KV head)
KINDS = [("same", BF, 64, 4), ("same", BF, 128, 8), ("same", F16, 128, 1), ("same", BF, 256, 3), ("same", F16, 64, 12),
         ("e4m3", BF, 128, 4), ("e4m3", F16, 256, 8), ("fp4", BF, 64, 8), ("fp4", F16, 128, 4), ("fp4", BF, 256, 2),
         ("same", F32, 64, 2), ("same", F32, 128, 9), ("same", F32, 256, 1)]
# (window, sinks): inside a page, on its border, one token, first tokens over several pages or none, meeting the window
WINDOWS = [(1, 0), (1, 1), (16, 0), (16, 16), (17, 4), (100, 4), (128, 33), (250, 100), (400, 0), (5, 300)]


def scales(cache, Hkv):
    return dict(k_scale=0.05, v_scale=0.07) if cache == "e4m3" else dict(k_scale=np.linspace(0.4, 1.3, Hkv), v_scale=np.linspace(0.9, 0.7, Hkv)) \
        if cache == "fp4" else {}


def lengths(W, K):
    return [0, 1, 15, 16, 17, max(W - 1, 1), W, W + 1, W + K, W + K + 1, W + 33, 700, 513]


@pytest.mark.parametrize("W,K", WINDOWS)
@pytest.mark.parametrize("cache,dtype,D,G", KINDS)
def test_decode(cache, dtype, D, G, W, K):
    Hkv = 2
    c = wc.make(lengths(W, K), Hkv * G, Hkv, D, W, K, dtype, cache, seed=W + K, **scales(cache, Hkv))
    g, want = wc.on_gpu(c), wc.reference(c)
    for part in (0, -1, 16, 48, -2, -8, BAL):
        wc.check(wc.run(c, g, part), want, "partition %d" % part)
        assert pa.pa_check_device_error(g.err) == (0, 0)
    wc.check(wc.run(c, g, 0, ws=False), want, "the library's workspace")


@pytest.mark.parametrize("cache,dtype,D,G", [("same", BF, 128, 4), ("same", F32, 64, 4), ("e4m3", BF, 128, 8), ("fp4", F16, 128, 4)])
def test_decode_alibi_and_layouts(cache, dtype, D, G):
    Hkv, W, K = 2, 90, 20
    slopes = np.linspace(0.01, 0.5, Hkv * G)
    for nhd in (False, True):
        if nhd and cache == "fp4":
            continue
        c = wc.make(lengths(W, K), Hkv * G, Hkv, D, W, K, dtype, cache, seed=3, alibi=slopes, nhd=nhd, **scales(cache, Hkv))
        g, want = wc.on_gpu(c), wc.reference(c)
        for part in (0, 32, -4, BAL):
            wc.check(wc.run(c, g, part), want, "alibi, partition %d, nhd %s" % (part, nhd))


NEWS = [1, 3, 0, 5, 1, 2, 40, 7]


@pytest.mark.parametrize("W,K", [(1, 0), (16, 16), (17, 4), (100, 33), (250, 100), (5, 300)])
@pytest.mark.parametrize("cache,dtype,D,G", KINDS)
def test_columns(cache, dtype, D, G, W, K):
    """Several new tokens on the decode kernels (a split asked for, or few columns)."""
    Hkv = 2
    lens = [1, 30, 40, 200, 700, W + 2, W + 45, 333]
    c = wc.make(lens, Hkv * G, Hkv, D, W, K, dtype, cache, nq=NEWS, seed=W + K, extra_rows=2, **scales(cache, Hkv))
    g, want = wc.on_gpu(c), wc.reference(c)
    n = sum(NEWS)
    for part in (32, -2):
        out = wc.run(c, g, part)
        assert bool(torch.isnan(out[n:]).all())  # rows of no sequence are left
        wc.check(out[:n], (want[0][:n], want[1][:n]), "partition %d" % part)
        assert pa.pa_check_device_error(g.err) == (0, 0)


@pytest.mark.parametrize("W,K", [(1, 0), (1, 20), (16, 16), (63, 1), (64, 64), (100, 4), (130, 70), (300, 0), (700, 200), (5, 300)])
@pytest.mark.parametrize("dtype,D,G", [(BF, 64, 4), (F16, 64, 8), (BF, 128, 4), (F16, 128, 8), (BF, 128, 1), (BF, 128, 3), (BF, 256, 4), (F16, 256, 1),
                                       (F16, 256, 12)])
def test_chunks(dtype, D, G, W, K):
    """Long chunks on the query-tile kernel: one and two tiles a CTA, chunks that end inside a tile, sequences
    without history, and of a single new token."""
    Hkv = 2
    news = [130, 1, 64, 0, 33, 200]
    lens = [130, 500, 300, 77, 900, 777]
    c = wc.make(lens, Hkv * G, Hkv, D, W, K, dtype, nq=news, seed=W + K, extra_rows=3)
    g, want = wc.on_gpu(c), wc.reference(c)
    n = sum(news)
    for part in (0, 128):
        out = wc.run(c, g, part)
        assert bool(torch.isnan(out[n:]).all())
        wc.check(out[:n], (want[0][:n], want[1][:n]), "partition %d" % part)
        assert pa.pa_check_device_error(g.err) == (0, 0)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunks_alibi_and_nhd(D):
    Hkv, G = 2, 4
    c = wc.make([300, 170, 600], Hkv * G, Hkv, D, 90, 20, BF, nq=[64, 170, 129], seed=8, alibi=np.linspace(0.01, 0.3, Hkv * G),
                nhd=True)
    g = wc.on_gpu(c)
    wc.check(wc.run(c, g), wc.reference(c))


@pytest.mark.parametrize("cache,dtype,D", [("same", BF, 128), ("e4m3", BF, 128), ("fp4", BF, 128), ("same", F32, 64)])
def test_a_window_that_holds_everything_is_the_plain_call(cache, dtype, D):
    c = wc.make([0, 5, 100, 257], 8, 2, D, 10 ** 6, 0, dtype, cache, seed=2, **scales(cache, 2))
    g = wc.on_gpu(c)
    want = torch.full_like(g.out, float("nan"))
    pa.pa_decode_opt(want, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, 2, g.k_scale, g.v_scale, g.stride)
    for W, K in ((c.width * 16, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, c.width * 16), (c.width * 16 - 4, 4)):
        c.W, c.K = W, K
        assert torch.equal(wc.run(c, g), want)


def test_many_sequences_of_every_length():
    """More units than CTAs at once, ordered by length; one query each, the plans' own choice."""
    lens = [int(x) for x in np.random.RandomState(0).randint(0, 900, 120)]
    for cache, dtype, D in (("same", BF, 64), ("fp4", BF, 128), ("e4m3", BF, 128)):
        c = wc.make(lens, 16, 8, D, 200, 7, dtype, cache, seed=1, **scales(cache, 8))
        g = wc.on_gpu(c)
        wc.check(wc.run(c, g), wc.reference(c), cache)


@pytest.mark.parametrize("nq", [None, [3, 1, 2], [70, 64, 65]])
def test_bad_blocks_and_lengths(nq):
    """A seen entry out of range, or a length beyond the table: that sequence writes nothing, its bit is set,
    and the others are right."""
    lens = [400, 300, 350]
    c = wc.make(lens, 8, 2, 128, 100, 4, BF, nq=nq, seed=4)
    want = wc.reference(c)
    starts = [0, 1, 2, 3] if nq is None else np.concatenate([[0], np.cumsum(nq)])
    for what, bit in (("block", pa.PA_DEVERR_BLOCK_RANGE), ("first", pa.PA_DEVERR_BLOCK_RANGE), ("length", pa.PA_DEVERR_SEQLEN_RANGE)):
        for part in (0, 16) if nq is None else (0,):
            g = wc.on_gpu(c)
            if what == "length":
                g.seq_lens[1] = c.width * 16 + 1
            else:
                g.block_table[1, 0 if what == "first" else (lens[1] - 1) // 16] = c.NB
            out = wc.run(c, g, part)
            for s in range(3):
                a, b = starts[s], starts[s + 1]
                if s == 1:
                    assert bool(torch.isnan(out[a:b]).all())
                else:
                    wc.check(out[a:b], (want[0][a:b], want[1][a:b]))
            assert pa.pa_check_device_error(g.err) == (-6, bit)
            g2 = wc.on_gpu(c)
            g2.ws = g.ws  # (the counters are back at zero)
            wc.check(wc.run(c, g2, part), want)


@pytest.mark.parametrize("nq,D", [(None, 128), ([70, 64, 65], 128), ([200, 130, 1], 128), ([70, 64, 65], 256), ([200, 130, 1], 64)])
def test_a_wait_that_gives_up(nq, D):
    c = wc.make([400, 300, 350], 8, 2, D, 100, 4, BF, nq=nq, seed=4)
    g = wc.on_gpu(c)
    out = wc.run(c, g, 0, first_wait_limit=-1)
    assert pa.pa_check_device_error(g.err) == (-8, pa.PA_DEVERR_WAIT_TIMEOUT)
    assert bool(torch.isnan(out).all())
    wc.check(wc.run(c, g), wc.reference(c))


@pytest.mark.parametrize("cache,dtype", [("same", BF), ("e4m3", BF), ("fp4", BF), ("same", F32)])
def test_workspace_size(cache, dtype):
    code = {"e4m3": pa.PA_FP8_E4M3, "fp4": pa.PA_FP4_E2M1}.get(cache, pa.PA_F32 if dtype is F32 else pa.PA_BF16)
    for nq, parts in ((None, (0, 16, 64, BAL, -1, -4)), ([3, 1], (0, 16, 64, -1))):
        c = wc.make([3000, 2500], 8, 2, 128, 600, 20, dtype, cache, nq=nq, seed=6, **scales(cache, 2))
        g, want = wc.on_gpu(c), wc.reference(c)
        for part in parts:
            need = pa.pa_decode_window_workspace_size(2, 8, 2, 128, c.width, code, 600, 20, 1 if nq is None else 3, part)
            g.ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
            wc.check(wc.run(c, g, part), want, "partition %d" % part)
            if need and part > 0:
                g.ws = g.ws[:need - 1]
                with pytest.raises(pa.PAError) as e:
                    wc.run(c, g, part)
                assert e.value.status == -4
        assert pa.pa_decode_window_workspace_size(2, 8, 2, 128, c.width, code, 600, 20, 1, -1) == 0


def test_side_streams_and_graphs():
    """Two calls at once, each with its own workspace on its own stream; captured and replayed with the
    lengths and tables of a later step."""
    c = wc.make([900, 40, 333], 8, 2, 128, 300, 4, BF, seed=7)
    d = wc.make([120, 870], 8, 2, 64, 100, 16, F16, seed=8)
    gc, gd = wc.on_gpu(c), wc.on_gpu(d)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, (x, g) in zip(streams, ((c, gc), (d, gd))):
            with torch.cuda.stream(st):
                wc.run(x, g, 32)
    torch.cuda.synchronize()
    wc.check(gc.out, wc.reference(c))
    wc.check(gd.out, wc.reference(d))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wc.run(c, gc, 32)
    later = wc.make([902, 42, 335], 8, 2, 128, 300, 4, BF, seed=9)
    assert (later.NB, later.width) == (c.NB, c.width)
    gl = wc.on_gpu(later)
    for name in ("k_cache", "v_cache", "q", "block_table", "seq_lens"):
        getattr(gc, name).copy_(getattr(gl, name))
    graph.replay()
    torch.cuda.synchronize()
    wc.check(gc.out, wc.reference(later))


def test_calls_of_different_shapes_follow_each_other():
    """The library's workspace between windowed, plain and accumulating calls of other shapes and splits."""
    cases = [wc.make([3000, 20, 1500], 8, 2, 128, 900, 4, BF, seed=1), wc.make([700] * 9, 32, 4, 64, 333, 0, F16, seed=2),
             wc.make([400, 2000], 8, 8, 128, 1000, 20, BF, "e4m3", seed=3, k_scale=0.05, v_scale=0.07)]
    on = [wc.on_gpu(c) for c in cases]
    want = [wc.reference(c) for c in cases]
    for part in (64, BAL, 0, 32, 512, BAL, 16):
        for c, g, w in zip(cases, on, want):
            wc.check(wc.run(c, g, part, ws=False), w, "partition %d" % part)
            full = wc.make([50, 300], 8, 2, 128, 10 ** 6, 0, BF, seed=4)
            gf = wc.on_gpu(full)
            pa.pa_decode_opt(gf.out, gf.q, gf.k_cache, gf.v_cache, gf.block_table, gf.seq_lens, full.scale, 2, partition_size=32)
            wc.check(gf.out, wc.reference(full))


QUANT = [("e4m3", BF, 128, 4), ("e4m3", F16, 256, 8), ("fp4", BF, 64, 8), ("fp4", F16, 128, 4), ("fp4", BF, 256, 2)]
CHUNK = ([130, 500, 300, 77, 900, 777, 101], [130, 1, 64, 0, 33, 200, 101])


def chunk_workspace(c, part=0):
    code = pa.PA_FP8_E4M3 if c.cache == "e4m3" else pa.PA_FP4_E2M1
    return pa.pa_decode_window_workspace_size(c.S, c.Hq, c.Hkv, c.D, c.width, code, c.W, c.K, max(c.nq), part)


@pytest.mark.parametrize("W,K", [(1, 0), (1, 20), (16, 16), (100, 4), (130, 70), (700, 200), (5, 300)])
@pytest.mark.parametrize("cache,dtype,D,G", QUANT)
def test_chunks_of_quantised_caches(cache, dtype, D, G, W, K):
    """Long chunks over E4M3 and 4-bit caches: widened into the library's workspace or the caller's (at 16 bytes off
    a 32-byte border too, which leaves the arrival counters at zero), and in columns where there is no room."""
    Hkv = 32 // G
    lens, news = CHUNK
    c = wc.make(lens, 32, Hkv, D, W, K, dtype, cache, nq=news, seed=W + K, extra_rows=3, **scales(cache, Hkv))
    g, want = wc.on_gpu(c), wc.reference(c)
    n = sum(news)
    want = want[0][:n], want[1][:n]
    need = chunk_workspace(c)
    assert need > 0 and chunk_workspace(c, -1) == need
    big = torch.zeros(need + 16, dtype=torch.uint8, device="cuda")
    for what, ws in (("library", None), ("exact", big[:need]), ("off by 16", big[16:]), ("columns", big[:need - 1])):
        if ws is not None:
            big.zero_()
            g.ws = ws
        for part in (0, -1):
            out = wc.run(c, g, part, ws=ws is not None)
            assert bool(torch.isnan(out[n:]).all())
            wc.check(out[:n], want, "%s, partition %d" % (what, part))
            assert pa.pa_check_device_error(g.err) == (0, 0)
        if ws is not None:
            counters = (c.S * Hkv * ((G * max(news) + 7) // 8) * 4 + 255) // 256 * 256
            assert not ws[:counters].any()
    wc.check(wc.run(c, g, 128, ws=False)[:n], want, "a split asked for")


@pytest.mark.parametrize("cache,dtype,D,G", QUANT)
def test_quantised_chunks_with_bias_layout_signs_and_bad_blocks(cache, dtype, D, G):
    Hkv = 32 // G
    lens, news = [300, 250, 600], [64, 250, 200]
    sc = dict(k_scale=np.resize([0.05, -0.03], Hkv), v_scale=np.resize([-0.07, 0.02, 0.06], Hkv))  # of both signs
    c = wc.make(lens, 32, Hkv, D, 90, 20, dtype, cache, nq=news, seed=8, alibi=np.linspace(0.01, 0.3, 32),
                nhd=cache == "e4m3", **sc)
    g = wc.on_gpu(c)
    wc.check(wc.run(c, g, ws=False), wc.reference(c), "ALiBi")
    c = wc.make(lens, 32, Hkv, D, 90, 20, dtype, cache, nq=news, seed=9, nhd=cache == "e4m3", **sc)
    g, want = wc.on_gpu(c), wc.reference(c)
    wc.check(wc.run(c, g, ws=False), want, "signs")
    g.block_table[1, 5] = c.NB
    out = wc.run(c, g, ws=False)
    assert pa.pa_check_device_error(g.err) == (-6, pa.PA_DEVERR_BLOCK_RANGE)
    assert bool(torch.isnan(out[64:314]).any())  # (its row tiles that see the page write nothing)
    for a, b in ((0, 64), (314, 514)):
        wc.check(out[a:b], (want[0][a:b], want[1][a:b]))
    g = wc.on_gpu(c)
    g.seq_lens[2] = -1
    out = wc.run(c, g, ws=False)
    assert pa.pa_check_device_error(g.err) == (-6, pa.PA_DEVERR_SEQLEN_RANGE)
    assert bool(torch.isnan(out[314:]).all())
    wc.check(out[:314], (want[0][:314], want[1][:314]))


def test_quantised_chunks_captured():
    """Captured with the library's workspace, replayed over other rows, tables and lengths, between other calls."""
    c = wc.make([300, 570], 32, 8, 128, 90, 20, BF, "e4m3", nq=[200, 320], seed=1, k_scale=0.05, v_scale=0.07)
    later = wc.make([303, 576], 32, 8, 128, 90, 20, BF, "e4m3", nq=[200, 320], seed=2, k_scale=0.05, v_scale=0.07)
    other = wc.make([500] * 6, 32, 4, 128, 200, 0, BF, "fp4", nq=[100] * 6, seed=3)
    assert (later.NB, later.width) == (c.NB, c.width)
    g, gl, go = wc.on_gpu(c), wc.on_gpu(later), wc.on_gpu(other)
    wc.run(c, g, ws=False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wc.run(c, g, ws=False)
    wc.check(wc.run(other, go, ws=False), wc.reference(other))  # (the workspace grows)
    for name in ("k_cache", "v_cache", "q", "block_table", "seq_lens"):
        getattr(g, name).copy_(getattr(gl, name))
    graph.replay()
    torch.cuda.synchronize()
    wc.check(g.out, wc.reference(later))
    wc.check(wc.run(other, go, ws=False), wc.reference(other))


def test_workspace_of_long_chunks_over_quantised_caches():
    """The size covers every call of at most max_query_len queries a sequence, and bounds itself."""
    size = lambda *a: pa.pa_decode_window_workspace_size(*a)
    for code in (pa.PA_FP8_E4M3, pa.PA_FP4_E2M1):
        a = size(64, 32, 8, 128, 512, code, 1024, 4, 512, 0)
        pages = (1024 + 511 + 14) // 16 + 1 + 1
        counters = (64 * 8 * (4 * 512 // 8) * 4 + 255) // 256 * 256
        assert a == counters + 2 * 64 * pages * 8 * 16 * 128 * 2 + 64 * 512 * 4
        assert size(64, 32, 8, 128, 512, code, 1024, 4, 512, -1) == a
        assert size(64, 32, 8, 128, 512, code, 1024, 4, 256, 0) < a
        assert size(256, 32, 8, 128, 4096, code, 8192, 4, 512, 0) < 1 << 28  # (past the limit: columns)
        for S in (1 << 17, 1 << 30):  # (products past 2^63)
            assert size(S, 32, 8, 256, 1 << 22, code, 1 << 25, 1 << 24, 512, -1) == 0
    assert size(64, 32, 8, 128, 512, pa.PA_BF16, 1024, 4, 512, 0) == 0


@pytest.mark.parametrize("cache,dtype,D,G", QUANT)
def test_quantised_chunks_of_padded_and_mixed_batches(cache, dtype, D, G):
    """A batch of one long chunk and many short ones (columns), and query rows padded far past the last sequence."""
    Hkv = 32 // G
    news = [200] + [1] * 30
    c = wc.make([400] + [150 + 7 * i for i in range(30)], 32, Hkv, D, 60, 17, dtype, cache, nq=news, seed=4,
                extra_rows=1100, **scales(cache, Hkv))
    g, want = wc.on_gpu(c), wc.reference(c)
    out = wc.run(c, g, ws=False)
    n = sum(news)
    wc.check(out[:n], (want[0][:n], want[1][:n]))
    assert bool(torch.isnan(out[n:]).all())
    c = wc.make([400] + [150 + 7 * i for i in range(30)], 32, Hkv, D, 60, 17, dtype, cache, nq=news, seed=4,
                **scales(cache, Hkv))
    wc.check(wc.run(c, wc.on_gpu(c), ws=False), wc.reference(c))
