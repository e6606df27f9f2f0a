"""Outputs whose rows share memory are refused (host only; no kernel is launched here): the rows are
written, or read and added to, by different blocks at once."""
import ctypes

import pytest

from test_abi import _t
from test_evict_host import _evict
from test_fp4_oracle import _accumulate

import paged_decode_attention_reshape_gb300 as pa

S, HQ, H, D, NB, MB, B = 3, 8, 2, 64, 16, 4, 20
W = MB * 16


@pytest.fixture(scope="module")
def L():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    return pa.lib()


def _strides(row):
    """Strides of [S, H, row]: shared, and (the last three) not."""
    return [[0, row, 1], [row, 0, 1], [0, 0, 1], [row, row, 1], [row - 1, S * row, 1], [H * row, row - 4, 1],
            [2 * row - 4, row, 1]], [[H * row, row, 1], [row, S * row, 1], [5 * H * row, 2 * row, 1]]


def test_weights(L):
    q, out, kc = _t([S, HQ, D], pa.PA_BF16), _t([S, HQ, D], pa.PA_BF16, ptr=0x20000), _t([NB, H, 16, D], pa.PA_BF16)
    bt, sl = _t([S, MB], pa.PA_I32), _t([S], pa.PA_I32)
    shared, apart = _strides(W)
    call = [_accumulate(L, out, q, kc, kc, bt, sl, H, _t([S, H, W], pa.PA_F32, ptr=p, strides=st))
            for p, st in [(0x10000, st) for st in shared] + [(0x10002, st) for st in apart]]
    assert call == [-1] * len(shared) + [-3] * len(apart)          # (-3: past this check, refused for the pointer)
    one = _t([1, 1, W], pa.PA_F32, ptr=0x10002, strides=[0, 0, 1])  # single rows share nothing
    assert _accumulate(L, _t([1, 4, D], pa.PA_BF16), _t([1, 4, D], pa.PA_BF16), _t([NB, 1, 16, D], pa.PA_BF16),
                       _t([NB, 1, 16, D], pa.PA_BF16), _t([1, MB], pa.PA_I32), _t([1], pa.PA_I32), 1, one) == -3


def test_evict(L):
    for name, row, ptr in (("kept", B, 0x20002), ("nw", W, 0x40002)):
        dt = pa.PA_I32 if name == "kept" else pa.PA_F32
        shared, apart = _strides(row)
        assert [_evict(L, **{name: _t([S, H, row], dt, ptr=ptr, strides=st)}) for st in shared] == [-1] * len(shared)
        assert [_evict(L, **{name: _t([S, H, row], dt, ptr=ptr, strides=st)}) for st in apart] == [-3] * len(apart)


def test_read_back(L):
    cache, slots = _t([NB, H, 16, D], pa.PA_BF16), _t([S], pa.PA_I64, ptr=0x10004)
    good = _t([S, H, D], pa.PA_BF16)
    shared, apart = _strides(D)
    for strides, status in [(st, -1) for st in shared] + [(st, -3) for st in apart]:
        bad = _t([S, H, D], pa.PA_BF16, strides=strides)
        for key, value in ((bad, good), (good, bad)):
            r = [ctypes.byref(x) for x in (key, value, cache, cache, slots)]
            assert L.pa_gather_cache(*r, None, None) == status
