"""Cache writes of nothing (host only; no kernel is launched here)."""
import ctypes

import pytest

from test_abi import _t

import paged_decode_attention_reshape_gb300 as pa


@pytest.fixture(scope="module")
def L():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    return pa.lib()


def _write(L, rows, cache, kv, slots):
    r = [ctypes.byref(x) for x in (rows, rows, cache, cache, slots)]
    return L.pa_reshape_and_cache(*r, kv, None, None, None, None)


KINDS = [(pa.PA_BF16, pa.PA_KV_AUTO), (pa.PA_FP8_E4M3, pa.PA_KV_FP8_E4M3), (pa.PA_FP4_E2M1, pa.PA_KV_FP4_E2M1)]


@pytest.mark.parametrize("held,kv", KINDS)
def test_no_heads_or_no_elements(L, held, kv):
    T, NB, D = 3, 4, 64
    page = (9 * D,) if held == pa.PA_FP4_E2M1 else (16, D)
    slots = _t([T], pa.PA_I64)
    assert _write(L, _t([T, 0, D], pa.PA_BF16), _t([NB, 0, *page], held), kv, slots) == 0
    if held != pa.PA_FP4_E2M1:
        assert _write(L, _t([T, 2, 0], pa.PA_BF16), _t([NB, 2, 16, 0], held), kv, slots) == -7
