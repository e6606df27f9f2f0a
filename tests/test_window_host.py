"""pa_decode_window and pa_attention_window without a GPU: refusals that come before any launch."""
import ctypes

import pytest

import paged_decode_attention_reshape_gb300 as pa
from test_abi import _t

S, HQ, HKV, D, NB, MB = 3, 8, 2, 128, 16, 40


@pytest.fixture(scope="module")
def L():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    return pa.lib()


def _args():
    return dict(out=_t([S, HQ, D], pa.PA_BF16, 0x20000), q=_t([S, HQ, D], pa.PA_BF16), kc=_t([NB, HKV, 16, D], pa.PA_BF16),
                vc=_t([NB, HKV, 16, D], pa.PA_BF16), starts=_t([S + 1], pa.PA_I32), bt=_t([S, MB], pa.PA_I32),
                sl=_t([S], pa.PA_I32), hkv=HKV, nq=4, window=64, sinks=4, opt=None)


def _call(L, chunk, a):
    p = {k: (ctypes.byref(v) if isinstance(v, ctypes.Structure) else v) for k, v in a.items()}
    if chunk:
        return L.pa_attention_window(p["out"], p["q"], p["kc"], p["vc"], p["starts"], p["bt"], p["sl"], 0.125, p["hkv"],
                                     p["nq"], p["window"], p["sinks"], p["opt"], None)
    return L.pa_decode_window(p["out"], p["q"], p["kc"], p["vc"], p["bt"], p["sl"], 0.125, p["hkv"], p["window"],
                              p["sinks"], p["opt"], None)


@pytest.mark.parametrize("chunk", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(window=0), -1), (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(window=-2 ** 31), -1),
    (dict(q=None), -1), (dict(hkv=3), -1), (dict(bt=_t([S, MB], pa.PA_I64)), -2), (dict(sl=_t([S + 1], pa.PA_I32)), -1),
    (dict(q=_t([S, HQ, D], pa.PA_F16)), -1), (dict(out=_t([S, HQ, D], pa.PA_BF16, 0x20008)), -3),
    (dict(kc=_t([NB, HKV, 16, 96], pa.PA_BF16), vc=_t([NB, HKV, 16, 96], pa.PA_BF16)), -1),
    (dict(kc=_t([NB, HKV, 8, D], pa.PA_BF16), vc=_t([NB, HKV, 8, D], pa.PA_BF16)), -7)])
def test_refusals(L, chunk, change, status):
    a = _args()
    a.update(change)
    assert _call(L, chunk, a) == status


def test_chunk_refusals(L):
    a = _args()
    a["starts"] = None
    assert _call(L, True, a) == -1
    a = _args()
    a["nq"] = 0
    assert _call(L, True, a) == -1
    o = pa.PaDecodeOptions()
    o.partition_size = pa.PA_PARTITION_BALANCED
    a = _args()
    a["opt"] = o
    assert _call(L, True, a) == -7


def test_nothing_to_do(L):
    a = _args()
    for k in ("out", "q"):
        a[k] = _t([0, HQ, D], pa.PA_BF16, 0)
    a["bt"], a["sl"] = _t([0, MB], pa.PA_I32), _t([0], pa.PA_I32)
    assert _call(L, False, a) == 0


def test_workspace_size_of_invalid_arguments(L):
    good = dict(num_seqs=4, num_heads=32, num_kv_heads=8, head_size=128, max_blocks_per_seq=1000,
                kv_dtype_code=pa.PA_BF16, window=512, sinks=4, max_query_len=1, partition_size=16)
    for change in (dict(num_heads=30), dict(window=0), dict(sinks=-1), dict(kv_dtype_code=99), dict(max_query_len=0),
                   dict(num_seqs=-1), dict(max_blocks_per_seq=-1), dict(num_heads=2 ** 20, max_query_len=2 ** 20)):
        assert pa.pa_decode_window_workspace_size(**{**good, **change}) == 0
