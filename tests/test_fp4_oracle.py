"""The oracle's 4-bit codec on the host, and the refusals of the calls that take 4-bit caches (no
kernel is launched here)."""
import ctypes

import numpy as np
import pytest

import oracle
from test_abi import _decode, _t, _write

import paged_decode_attention_reshape_gb300 as pa


@pytest.fixture(scope="module")
def L():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    return pa.lib()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_page_places_cover_the_page_once(D):
    assert np.array_equal(np.sort(oracle.fp4_place(D).ravel()), np.arange(9 * D))


def test_codes_are_the_nearest_values():
    rng = np.random.RandomState(1)
    x = (rng.randn(40, 2, 64) * np.exp(rng.randn(40, 2, 1) * 3)).astype(np.float32)
    code, sg = oracle.fp4_quantize(x, 1.0)
    v = oracle.fp4_values(code, sg)
    s = np.repeat(oracle.e4m3_decode(sg), 16, -1)
    cand = np.concatenate([-oracle.E2M1_VALUES[::-1], oracle.E2M1_VALUES]) * s[..., None]
    best = np.abs(cand - x[..., None].astype(np.float64)).min(-1)
    assert (np.abs(v - x) <= best * (1 + 1e-6)).all()
    # the group's largest element is within one sixth of a step of the scale's rounding of 6 sg
    top = np.abs(x).reshape(40, 2, 4, 16).max(-1)
    e = oracle.e4m3_decode(sg)
    ok = (np.abs(e - top / 6) <= np.maximum(e / 16, 2.0 ** -10)) | (top / 6 < 2.0 ** -9) | (top / 6 > 448)
    assert ok.all()


def test_special_groups():
    x = np.zeros((1, 1, 64), dtype=np.float32)
    x[0, 0, 3] = np.nan
    x[0, 0, 16] = np.inf
    x[0, 0, 33] = -1e-6
    code, sg = oracle.fp4_quantize(x, 1.0)
    assert sg[0, 0].tolist() == [0x7F, 0x7E, 0x01, 0x01]
    assert not code[0, 0, :16].any() and code[0, 0, 16] == 7 and code[0, 0, 33] == 8 and not code[0, 0, 48:].any()


def test_write_refusals(L):
    T, H, D, NB = 4, 2, 64, 8
    key, sm = _t([T, H, D], pa.PA_BF16), _t([T], pa.PA_I64)
    page = _t([NB, H, 9 * D], pa.PA_FP4_E2M1)
    kv = pa.PA_KV_FP4_E2M1
    empty = _t([0, H, D], pa.PA_BF16)
    assert _write(L, empty, empty, page, page, _t([0], pa.PA_I64), kv) == 0
    assert _write(L, key, key, page, page, sm, pa.PA_KV_AUTO) == -2                    # mode and cache differ
    assert _write(L, key, key, page, page, sm, pa.PA_KV_FP8_E4M3) == -2
    assert _write(L, key, key, _t([NB, H, 16, D], pa.PA_BF16), _t([NB, H, 16, D], pa.PA_BF16), sm, kv) == -2
    assert _write(L, key, key, _t([NB, H, 16, D], pa.PA_FP4_E2M1), page, sm, kv) == -1  # pages have rank 3
    assert _write(L, key, key, _t([NB, H, 9 * 96], pa.PA_FP4_E2M1), _t([NB, H, 9 * 96], pa.PA_FP4_E2M1), sm, kv) == -7
    assert _write(L, key, key, _t([NB, H, 9 * 128], pa.PA_FP4_E2M1), _t([NB, H, 9 * 128], pa.PA_FP4_E2M1), sm, kv) == -1
    assert _write(L, key, key, page, _t([NB, H + 1, 9 * D], pa.PA_FP4_E2M1), sm, kv) == -1
    assert _write(L, key, key, _t([NB, H, 9 * D], pa.PA_FP4_E2M1, ptr=0x10008), page, sm, kv) == -3
    assert _write(L, key, key, _t([NB, H, 9 * D], pa.PA_FP4_E2M1, strides=[H * 9 * D + 8, 9 * D, 1]), page, sm, kv) == -3
    assert _write(L, key, key, _t([NB, H, 9 * D], pa.PA_FP4_E2M1, strides=[H * 18 * D, 18 * D, 2]), page, sm, kv) == -1
    assert _write(L, _t([T, H, D], pa.PA_FP4_E2M1), _t([T, H, D], pa.PA_FP4_E2M1), page, page, sm, kv) == -2
    f8 = _t([T, H, D], pa.PA_FP8_E4M3)
    assert _write(L, f8, f8, page, page, sm, kv) == -2


def _gather(L, key, val, kc, vc, sm, opt=None):
    return L.pa_gather_cache(ctypes.byref(key), ctypes.byref(val), ctypes.byref(kc), ctypes.byref(vc),
                             ctypes.byref(sm), opt, None)


def test_gather_refusals(L):
    T, H, D, NB = 4, 2, 64, 8
    key, sm = _t([T, H, D], pa.PA_BF16), _t([T], pa.PA_I64)
    page = _t([NB, H, 9 * D], pa.PA_FP4_E2M1)
    bf = _t([NB, H, 16, D], pa.PA_BF16)
    empty = _t([0, H, D], pa.PA_BF16)
    assert _gather(L, empty, empty, page, page, _t([0], pa.PA_I64)) == 0
    assert _gather(L, key, _t([T, H, D], pa.PA_F16), page, page, sm) == -1
    assert _gather(L, _t([T, H, D], pa.PA_FP8_E4M3), _t([T, H, D], pa.PA_FP8_E4M3), page, page, sm) == -2
    assert _gather(L, _t([T, H, D], pa.PA_F16), _t([T, H, D], pa.PA_F16), bf, bf, sm) == -2   # no conversion
    assert _gather(L, key, key, page, page, _t([T], pa.PA_I32)) == -2
    assert _gather(L, key, key, page, page, _t([T + 1], pa.PA_I64)) == -1
    assert _gather(L, _t([T, H + 1, D], pa.PA_BF16), _t([T, H + 1, D], pa.PA_BF16), page, page, sm) == -1
    assert _gather(L, _t([T, H, D], pa.PA_BF16, ptr=0x10004), key, page, page, sm) == -3
    assert _gather(L, _t([T, H, D], pa.PA_BF16, strides=[H * D + 4, D, 1]), key, page, page, sm) == -3
    assert _gather(L, _t([T, H, D], pa.PA_BF16, ptr=0), key, page, page, sm) == -1
    b24 = _t([NB, H, 16, 24], pa.PA_BF16)
    assert _gather(L, _t([T, H, 24], pa.PA_BF16), _t([T, H, 24], pa.PA_BF16), b24, b24, sm) == -7
    o = pa.PaWriteOptions()
    o.scale_stride = -1
    assert _gather(L, key, key, page, page, sm, ctypes.byref(o)) == -1


def test_copy_blocks_refusals(L):
    NB, H, D = 4, 2, 64
    pairs = _t([1, 2], pa.PA_I64)

    def copy(k, v):
        return L.pa_copy_blocks(ctypes.byref(k), ctypes.byref(v), ctypes.byref(pairs), None, None)
    page = _t([NB, H, 9 * D], pa.PA_FP4_E2M1)
    assert copy(_t([NB, H, 16, D], pa.PA_FP4_E2M1), _t([NB, H, 16, D], pa.PA_FP4_E2M1)) == -1
    assert copy(page, _t([NB, H, 16, D], pa.PA_BF16)) == -1
    assert copy(page, _t([NB, H, 9 * D], pa.PA_FP4_E2M1, ptr=0x10008)) == -3


def _accumulate(L, out, q, kc, vc, bt, sl, hkv, w, opt=None):
    return L.pa_decode_accumulate(ctypes.byref(out), ctypes.byref(q), ctypes.byref(kc), ctypes.byref(vc),
                                  ctypes.byref(bt), ctypes.byref(sl), 0.1, hkv, None if w is None else ctypes.byref(w),
                                  None if opt is None else ctypes.byref(opt), None)


def test_decode_and_accumulate_refusals(L):
    S, Hq, H, D, NB, MB = 3, 8, 2, 128, 16, 4
    q, out = _t([S, Hq, D], pa.PA_BF16), _t([S, Hq, D], pa.PA_BF16, ptr=0x20000)
    page, bt, sl = _t([NB, H, 9 * D], pa.PA_FP4_E2M1), _t([S, MB], pa.PA_I32), _t([S], pa.PA_I32)
    assert _decode(L, _t([S, Hq, D], pa.PA_F32), _t([S, Hq, D], pa.PA_F32), page, page, bt, sl, H) == -2
    assert _decode(L, _t([S, Hq, 64], pa.PA_BF16), _t([S, Hq, 64], pa.PA_BF16), page, page, bt, sl, H) == -1
    assert _decode(L, out, q, page, _t([NB, H, 16, D], pa.PA_BF16), bt, sl, H) == -1
    assert _decode(L, out, q, _t([NB, H, 16, D], pa.PA_FP4_E2M1), page, bt, sl, H) == -1
    assert _decode(L, out, q, page, page, bt, sl, 3) == -1
    none_at_all = _t([0, H, 9 * D], pa.PA_FP4_E2M1)
    assert _decode(L, out, q, none_at_all, none_at_all, bt, sl, H) == -1            # no block to stand in
    wide = _t([NB, H, 9 * D], pa.PA_FP4_E2M1, strides=[1 << 32, 9 * D, 1])
    assert _decode(L, out, q, wide, page, bt, sl, H) == -7                          # block stride of 4 GiB
    w = _t([S, H, MB * 16], pa.PA_F32)
    none = pa.PaDecodeOptions()
    assert _accumulate(L, out, q, page, page, bt, sl, H, None) == -1
    assert _accumulate(L, out, q, page, page, bt, sl, H, _t([S, H, MB * 16], pa.PA_BF16)) == -2
    assert _accumulate(L, out, q, page, page, bt, sl, H, _t([S, H, MB * 16 - 1], pa.PA_F32)) == -1
    assert _accumulate(L, out, q, page, page, bt, sl, H, _t([S, H + 1, MB * 16], pa.PA_F32)) == -1
    assert _accumulate(L, out, q, page, page, bt, sl, H, _t([S, H, MB * 16], pa.PA_F32, ptr=0)) == -1
    assert _accumulate(L, out, q, page, page, bt, sl, H, _t([S, H, MB * 16], pa.PA_F32, ptr=0x10002)) == -3
    assert _accumulate(L, out, q, page, page, bt, sl, H, _t([S, H, MB * 16], pa.PA_F32, strides=[999, 99, 2])) == -1
    for P in (-2, -8):
        none.partition_size = P
        assert _accumulate(L, out, q, page, page, bt, sl, H, w, none) == -7
    empty = _t([0, Hq, D], pa.PA_BF16)
    assert _accumulate(L, empty, empty, page, page, _t([0, MB], pa.PA_I32), _t([0], pa.PA_I32), H,
                       _t([0, H, MB * 16], pa.PA_F32)) == 0


def test_accumulate_workspace_size(L):
    size = pa.pa_decode_accumulate_workspace_size
    # unsplit: one log-sum per (sequence, head), one score per (sequence, KV head, token, column)
    assert size(4, 32, 8, 128, 64, -1) == size(4, 32, 8, 128, 64, 0) == 4 * 32 * 4 + 4 * 8 * 64 * 16 * 4 * 4
    assert size(1, 3, 1, 64, 2, 0) == 256 + 2 * 16 * 4 * 4                   # 3 columns are kept as 4
    assert size(1, 9, 1, 64, 2, 0) == 256 + 2 * 2 * 16 * 8 * 4               # 9 heads: two groups of 8
    split = pa.pa_decode_workspace_size(4, 32, 8, 128, 64, 256)
    assert size(4, 32, 8, 128, 64, 256) == (split + 255) // 256 * 256 + size(4, 32, 8, 128, 64, 0)
    assert size(4, 30, 8, 128, 64, 0) == 0 and size(4, 32, 8, 128, 64, -2) == 0


def test_plan_of_a_4_bit_cache(L):
    B = pa.PA_PARTITION_BALANCED
    # many units: over the warps of a resident wave (152 SMs x 2 CTAs x 8 warps over 8 head rows)
    assert pa.pa_decode_plan(256, 32, 8, 128, 256, pa.PA_FP4_E2M1, 152, 0) == (B, 152 * 16 // 8)
    # fewer: whole, unless asked
    assert pa.pa_decode_plan(128, 64, 8, 128, 512, pa.PA_FP4_E2M1, 152, 0) == (0, 1)
    assert pa.pa_decode_plan(128, 64, 8, 128, 512, pa.PA_FP4_E2M1, 152, B) == (B, 152 * 16 // 8)
    # few long ones: over CTAs
    assert pa.pa_decode_plan(4, 32, 8, 128, 8192, pa.PA_FP4_E2M1, 152, 0)[0] == B
    # few short ones: fixed partitions, of 512 tokens at least, or none
    P, n = pa.pa_decode_plan(1, 32, 8, 128, 512, pa.PA_FP4_E2M1, 152, 0)
    assert P == 512 and n == 16
    assert pa.pa_decode_plan(2, 4, 4, 64, 3, pa.PA_FP4_E2M1, 152, 0) == (0, 1)
    # batches past the balanced split's limit: unsplit
    assert pa.pa_decode_plan(4096, 32, 8, 128, 256, pa.PA_FP4_E2M1, 152, 0) == (0, 1)
    assert pa.pa_decode_plan(128, 64, 8, 128, 512, pa.PA_FP4_E2M1, 152, 512) == (512, 16)
