"""Windowed decodes of more units than CTAs fit at once: every tensor-core kernel in CTAs of half the warps, with
and without the longest-first order, for short windows (any number of units) and for as many units as
twice the CTAs hold (longer windows).  And the calls of one input repeat themselves bit for bit."""
import numpy as np
import pytest
import torch

import window_cases as wc

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
KINDS = [("same", dt, D) for dt in (BF, F16) for D in (64, 128, 256)] \
    + [("e4m3", dt, D) for dt in (BF, F16) for D in (128, 256)] + [("fp4", dt, D) for dt in (BF, F16) for D in (64, 128, 256)]


def scales(cache, Hkv):
    n = np.linspace(0.5, 1.3, Hkv)
    return dict(k_scale=0.05, v_scale=0.07) if cache == "e4m3" else dict(k_scale=n, v_scale=n[::-1]) if cache == "fp4" else {}


def check(S, Hkv, G, longest, W, K, cache, dtype, D):
    rng = np.random.RandomState(S)
    lens = rng.randint(0, 90, S)
    lens[rng.permutation(S)[:6]] = [longest, longest - 1, W, W + 1, 0, longest // 2]
    c = wc.make([int(n) for n in lens], Hkv * G, Hkv, D, W, K, dtype, cache, seed=S, **scales(cache, Hkv))
    g, want = wc.on_gpu(c), wc.reference(c)
    wc.check(wc.run(c, g), want, "%d x %d" % (S, Hkv))
    first = g.out.clone()
    for _ in range(3):
        assert torch.equal(wc.run(c, g).view(torch.int16), first.view(torch.int16))


# An SM takes 1 to 6 CTAs of whole warps (152 to 912 units in all)
@pytest.mark.parametrize("cache,dtype,D", KINDS)
def test_short_windows(cache, dtype, D):
    check(120, 16, 1, 200, 60, 5, cache, dtype, D)   # (at most 128 sequences: ordered by length)
    check(240, 8, 2, 200, 33, 0, cache, dtype, D)


@pytest.mark.parametrize("S", [38, 75, 113])  # 304, 600 and 904 units: each holder of 1 to 6 CTAs meets one of them
@pytest.mark.parametrize("cache,dtype,D", KINDS)
def test_longer_windows(cache, dtype, D, S):
    check(S, 8, 3, 700, 420, 4, cache, dtype, D)


@pytest.mark.parametrize("dtype,D", [(BF, 64), (BF, 128), (F16, 128), (BF, 256)])
def test_chunks_repeat_themselves(dtype, D):
    c = wc.make([700, 333, 520, 130], 8, 2, D, 150, 20, dtype, nq=[333, 64, 1, 130], seed=2)
    g = wc.on_gpu(c)
    wc.check(wc.run(c, g), wc.reference(c))
    first = g.out.clone()
    for _ in range(20):
        assert torch.equal(wc.run(c, g).view(torch.int16), first.view(torch.int16))
