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

