"""Arrays and words off their element's size are refused (host only; no kernel is launched here): the
kernels read them element by element, and a misaligned address is a fault."""
import ctypes

import pytest

from test_abi import _t
from test_evict_host import _evict
from test_fp4_oracle import _accumulate

import paged_decode_attention_reshape_gb300 as pa

S, HQ, H, D, NB, MB, B = 3, 8, 2, 64, 16, 4, 20
I32, I64, F32, BF16 = pa.PA_I32, pa.PA_I64, pa.PA_F32, pa.PA_BF16


@pytest.fixture(scope="module")
def L():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    return pa.lib()


def refs(*tensors):
    return [None if t is None else ctypes.byref(t) for t in tensors]


def _decode(L, opt=None, bt=_t([S, MB], I32), sl=_t([S], I32), w=None):
    q, out, kc = _t([S, HQ, D], BF16), _t([S, HQ, D], BF16, ptr=0x20000), _t([NB, H, 16, D], BF16)
    if w is not None:
        return _accumulate(L, out, q, kc, kc, bt, sl, H, w, opt)
    return L.pa_decode_opt(*refs(out, q, kc, kc, bt, sl), 0.1, H, *refs(opt), None)


def test_decode(L):
    assert _decode(L, bt=_t([S, MB], I32, ptr=0x10002)) == -3
    assert _decode(L, sl=_t([S], I32, ptr=0x10001)) == -3
    assert _decode(L, w=_t([S, H, MB * 16], F32, ptr=0x10002)) == -3
    for field in ("k_scale", "v_scale", "alibi_slopes", "device_error"):
        o = pa.PaDecodeOptions()
        setattr(o, field, 0x10002)
        assert _decode(L, o) == -3


def test_varlen_and_step(L):
    q, out, kc = _t([S, HQ, D], BF16), _t([S, HQ, D], BF16, ptr=0x20000), _t([NB, H, 16, D], BF16)
    bt, sl, odd = _t([S, MB], I32), _t([S], I32), _t([S + 1], I32, ptr=0x10002)
    assert L.pa_attention_varlen(*refs(out, q, kc, kc, odd, bt, sl), 0.1, H, 1, None, None) == -3
    rows = _t([S, H, D], BF16)
    step = refs(out, q, rows, rows, kc, kc)
    assert L.pa_decode_step(*step, *refs(_t([S], I64), odd, bt, sl), 0.1, H, None, None) == -3


@pytest.mark.parametrize("held,kv", [(BF16, pa.PA_KV_AUTO), (pa.PA_FP4_E2M1, pa.PA_KV_FP4_E2M1)])
def test_write_and_read_back(L, held, kv):
    rows = _t([S, H, D], BF16)
    cache = _t([NB, H, 9 * D], held) if held == pa.PA_FP4_E2M1 else _t([NB, H, 16, D], held)
    slots, odd = _t([S], I64), _t([S], I64, ptr=0x10004)
    args = refs(rows, rows, cache, cache)
    assert L.pa_reshape_and_cache_opt(*args, *refs(odd), kv, None, None) == -3
    assert L.pa_gather_cache(*args, *refs(odd), None, None) == -3
    for field in ("k_scale", "v_scale", "device_error"):
        o = pa.PaWriteOptions()
        setattr(o, field, 0x10001)
        assert L.pa_reshape_and_cache_opt(*args, *refs(slots), kv, *refs(o), None) == -3
        assert L.pa_gather_cache(*args, *refs(slots, o), None) == -3


def test_evict_and_block_copy(L):
    W = MB * 16
    for name, t in (("bt", _t([S, MB], I32, ptr=0x10002)), ("sl", _t([S], I32, ptr=0x10001)),
                    ("w", _t([S, H, W], F32, ptr=0x10002)), ("kept", _t([S, H, B], I32, ptr=0x20002)),
                    ("nl", _t([S], I32, ptr=0x30003)), ("nw", _t([S, H, W], F32, ptr=0x40002))):
        assert _evict(L, **{name: t}) == -3
    kc = _t([NB, H, 16, D], BF16)
    assert L.pa_copy_blocks(*refs(kc, kc, _t([1, 2], I64, ptr=0x10004)), None, None) == -3
