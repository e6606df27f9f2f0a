"""The longest tables and weight rows that the accumulating decode and the eviction take: their kernels
count tokens in 32 bits, past the last one by up to a stride (host only; no kernel is launched here)."""

import pytest

from test_abi import _t
from test_evict_host import _evict
from test_fp4_oracle import _accumulate

import paged_decode_attention_reshape_gb300 as pa

TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    return pa.lib()


def test_accumulate(L):
    """Last token 2^31 - 17, stride 65535 x 1024 tokens: the next position does not fit."""
    S, Hq, H, D, NB = 1, 2, 1, 64, 4
    q, out, sl = _t([S, Hq, D], pa.PA_BF16), _t([S, Hq, D], pa.PA_BF16, ptr=0x20000), _t([S], pa.PA_I32)
    kc = _t([NB, H, 16, D], pa.PA_BF16)
    for MB in (TOP // 16, 2 ** 26 + 1):
        assert _accumulate(L, out, q, kc, kc, _t([S, MB], pa.PA_I32), sl, H, _t([S, H, TOP], pa.PA_F32)) == -7


def test_evict(L):
    S, H = 3, 2
    for W in (TOP, TOP - 1, TOP - 4095):
        w, nw = _t([S, H, W], pa.PA_F32), _t([S, H, W], pa.PA_F32, ptr=0x40000)
        assert _evict(L, w=w, nw=nw) == -7
        assert _evict(L, w=w, nw=nw, bt=_t([S, W // 16], pa.PA_I32)) == -7
