"""Rotary positions without a GPU: the frequency table, and every refusal of pa_rotary and
pa_rotary_and_cache (host checks that come before any launch)."""
import ctypes
import math

import pytest
import torch

import paged_decode_attention_reshape_gb300 as pa
from test_abi import _t


@pytest.fixture(scope="module")
def L():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    return pa.lib()


def turns(table):
    return torch.tensor([(f % 2 ** 64) / 2.0 ** 64 for f in table.tolist()], dtype=torch.float64)


@pytest.mark.parametrize("R,base", [(64, 10000.0), (128, 500000.0), (16, 3.7), (2, 10000.0)])
def test_frequencies_are_turns_per_position(L, R, base):
    want = torch.tensor([base ** (-2.0 * i / R) / (2 * math.pi) for i in range(R // 2)], dtype=torch.float64)
    # pow, a division and the conversion to 2^-64: a few 2^-53 of the value
    assert torch.allclose(turns(pa.pa_rotary_frequencies(R, base)), want, rtol=2e-15, atol=2.0 ** -64)


def test_scaled_frequencies(L):
    R, base, s, L0 = 128, 10000.0, 8.0, 4096.0
    plain = turns(pa.pa_rotary_frequencies(R, base))
    linear = turns(pa.pa_rotary_frequencies(R, base, pa.PA_ROTARY_LINEAR, s))
    assert torch.allclose(linear, plain / s, rtol=2e-15, atol=2.0 ** -63)
    based = turns(pa.pa_rotary_frequencies(R, base, pa.PA_ROTARY_BASE, s))
    assert based[0] == plain[0]
    assert abs(based[-1] * s / plain[-1] - 1) < 1e-13  # the slowest pair slows by the factor
    parts = turns(pa.pa_rotary_frequencies(R, base, pa.PA_ROTARY_PARTS, s, L0, 1.0, 32.0))
    n = L0 * plain
    assert bool((parts[n >= 32] == plain[n >= 32]).all()) and int((n >= 32).sum()) > 0
    assert torch.allclose(parts[n <= 1], plain[n <= 1] / s, rtol=2e-15, atol=2.0 ** -63) and int((n <= 1).sum()) > 0
    mid = (n > 1) & (n < 32)
    keep = (n - 1) / 31
    assert torch.allclose(parts[mid], (plain * keep + plain / s * (1 - keep))[mid], rtol=1e-14, atol=0)


def test_whole_turns_are_dropped(L):
    # base below 1: a pair that turns more than once per position keeps only the part
    base, R = 1e-3, 8
    theta = [base ** (-2.0 * i / R) for i in range(R // 2)]
    want = torch.tensor([math.fmod(t / (2 * math.pi), 1.0) for t in theta], dtype=torch.float64)
    assert torch.allclose(turns(pa.pa_rotary_frequencies(R, base)), want, rtol=0, atol=1e-13)


@pytest.mark.parametrize("args", [
    (7, 10000.0, 0, 1, 0, 1, 32), (-2, 10000.0, 0, 1, 0, 1, 32), (64, 0.0, 0, 1, 0, 1, 32),
    (64, -5.0, 0, 1, 0, 1, 32), (64, math.inf, 0, 1, 0, 1, 32), (64, math.nan, 0, 1, 0, 1, 32),
    (64, 10000.0, 4, 1, 0, 1, 32), (64, 10000.0, -1, 1, 0, 1, 32), (64, 10000.0, 1, 0.0, 0, 1, 32),
    (64, 10000.0, 1, math.nan, 0, 1, 32), (2, 10000.0, 2, 8.0, 0, 1, 32), (64, 10000.0, 3, 8.0, 0.0, 1, 32),
    (64, 10000.0, 3, 8.0, 4096.0, 32, 32), (64, 10000.0, 3, 8.0, 4096.0, 32, 1),
    (64, 10000.0, 3, 8.0, 4096.0, -1, 32), (64, 10000.0, 3, 8.0, 4096.0, 1, math.inf),
    (64, 1e-300, 2, 1e300, 0, 1, 32)])
def test_frequency_arguments_refused(L, args):
    with pytest.raises(pa.PAError) as e:
        pa.pa_rotary_frequencies(*args)
    assert e.value.status == -1


def test_no_pairs(L):
    assert pa.pa_rotary_frequencies(0).numel() == 0
    assert L.pa_rotary_frequencies(64, 10000.0, 0, 1.0, 0.0, 1.0, 32.0, None) == -1


T, HQ, HKV, D, NB = 5, 4, 2, 128, 3


def _args(cached):
    a = dict(q_out=_t([T, HQ, D], pa.PA_BF16, 0x100000), q=_t([T, HQ, D], pa.PA_BF16, 0x200000),
             key=_t([T, HKV, D], pa.PA_BF16, 0x300000), positions=_t([T], pa.PA_I64, 0x400000),
             frequencies=_t([D // 2], pa.PA_I64, 0x500000), q_weight=_t([D], pa.PA_BF16, 0x600000),
             k_weight=_t([D], pa.PA_F32, 0x700000), opt=pa.PaRotaryOptions())
    if cached:
        a.update(value=_t([T, HKV, D], pa.PA_BF16, 0x800000), k_cache=_t([NB, HKV, 16, D], pa.PA_BF16, 0x900000),
                 v_cache=_t([NB, HKV, 16, D], pa.PA_BF16, 0xA00000), slots=_t([T], pa.PA_I64, 0xB00000),
                 kv_dtype=pa.PA_KV_AUTO)
    else:
        a.update(k_out=_t([T, HKV, D], pa.PA_BF16, 0xC00000))
    return a


def _call(L, a):
    p = {k: (ctypes.byref(v) if isinstance(v, ctypes.Structure) else v) for k, v in a.items()}
    if "slots" in a:
        return L.pa_rotary_and_cache(p["q_out"], p["q"], p["key"], p["value"], p["k_cache"], p["v_cache"],
                                     p["positions"], p["slots"], p["frequencies"], p["q_weight"], p["k_weight"],
                                     p["kv_dtype"], p["opt"], None)
    return L.pa_rotary(p["q_out"], p["q"], p["k_out"], p["key"], p["positions"], p["frequencies"], p["q_weight"],
                       p["k_weight"], p["opt"], None)


def _option(**kw):
    o = pa.PaRotaryOptions()
    for k, v in kw.items():
        setattr(o, k, v)
    return o


B16 = pa.PA_BF16
COMMON = [
    (dict(q=None), -1), (dict(q_out=None), -1), (dict(q=None, q_out=None, q_weight=_t([D], B16)), -1),
    (dict(q=_t([T, HQ, D], pa.PA_F16)), -1),                                   # q_out of another type
    (dict(key=_t([T, HKV, D], pa.PA_F16)), -1), (dict(key=_t([T + 1, HKV, D], B16)), -1),
    (dict(q=_t([T, HQ, D], pa.PA_I32), q_out=_t([T, HQ, D], pa.PA_I32)), -2),
    (dict(q=_t([T, HQ, D], B16, strides=[HQ * D, D, 2])), -1),                  # innermost stride
    (dict(q_out=_t([T, HQ, D], B16, strides=[0, D, 1])), -1),                  # rows that share memory
    (dict(q_out=_t([T, HQ, D], B16, strides=[HQ * D, D // 2, 1])), -1),
    (dict(q_out=_t([T, HQ, D], B16, ptr=0x200000, strides=[2 * HQ * D, D, 1])), -1),  # in place, other strides
    (dict(q=_t([T, HQ, D], B16, ptr=0x200008)), -3), (dict(q=_t([T, HQ, D], B16, strides=[HQ * D + 4, D, 1])), -3),
    (dict(q=_t([T, HQ, D], B16, ptr=0)), -1), (dict(q_out=_t([T, HQ, D], B16, ptr=0)), -1),
    (dict(frequencies=_t([D // 2 + 8], pa.PA_I64)), -1), (dict(frequencies=_t([12], pa.PA_I64)), -7),
    (dict(frequencies=_t([64], pa.PA_I32)), -2), (dict(frequencies=_t([64], pa.PA_I64, ptr=0)), -1),
    (dict(frequencies=_t([64], pa.PA_I64, ptr=0x500004)), -3), (dict(frequencies=_t([64], pa.PA_I64, strides=[2])), -1),
    (dict(positions=None), -1), (dict(positions=_t([T], pa.PA_F32)), -2), (dict(positions=_t([T + 1], pa.PA_I64)), -1),
    (dict(positions=_t([T], pa.PA_I64, strides=[2])), -1), (dict(positions=_t([T], pa.PA_I64, ptr=0)), -1),
    (dict(positions=_t([T], pa.PA_I64, ptr=0x400004)), -3), (dict(positions=_t([T], pa.PA_I32, ptr=0x400002)), -3),
    (dict(q_weight=_t([D - 16], B16)), -1), (dict(q_weight=_t([D], pa.PA_F16)), -2), (dict(k_weight=_t([D], B16, ptr=0)), -1),
    (dict(k_weight=_t([D], pa.PA_F32, ptr=0x700002)), -3), (dict(k_weight=_t([D], B16, strides=[2])), -1),
    (dict(opt=_option(eps=-1e-6)), -1), (dict(opt=_option(eps=math.nan)), -1), (dict(opt=_option(eps=math.inf)), -1),
    (dict(opt=_option(scale_stride=-1)), -1),
]


@pytest.mark.parametrize("cached", [False, True])
@pytest.mark.parametrize("i", range(len(COMMON)))
def test_refusals(L, cached, i):
    change, status = COMMON[i]
    a = _args(cached)
    a.update(change)
    assert _call(L, a) == status


@pytest.mark.parametrize("change,status", [
    (dict(k_out=None), -1), (dict(key=None), -1),
    (dict(k_out=_t([T, HKV, D], B16, strides=[HKV * D, 0, 1])), -1),
    (dict(k_out=_t([T, HKV + 1, D], B16)), -1)])
def test_refusals_of_rows(L, change, status):
    a = _args(False)
    a.update(change)
    assert _call(L, a) == status


@pytest.mark.parametrize("change,status", [
    (dict(key=None), -1), (dict(value=None), -1), (dict(slots=None), -1), (dict(k_cache=None), -1),
    (dict(value=_t([T, HKV, D], pa.PA_F16)), -1), (dict(value=_t([T, HKV + 1, D], B16)), -1),
    (dict(slots=_t([T], pa.PA_I32)), -2), (dict(slots=_t([T + 1], pa.PA_I64)), -1), (dict(slots=_t([T], pa.PA_I64, ptr=0)), -1),
    (dict(slots=_t([T], pa.PA_I64, ptr=0xB00004)), -3),
    (dict(kv_dtype=7), -1), (dict(kv_dtype=pa.PA_KV_FP8_E4M3), -2), (dict(kv_dtype=pa.PA_KV_FP4_E2M1), -2),
    (dict(k_cache=_t([NB, HKV, 16, D], pa.PA_F16), v_cache=_t([NB, HKV, 16, D], pa.PA_F16)), -2),
    (dict(k_cache=_t([NB, HKV, 16, 64], B16), v_cache=_t([NB, HKV, 16, 64], B16)), -1),
    (dict(k_cache=_t([NB, HKV, 8, D], B16), v_cache=_t([NB, HKV, 8, D], B16)), -7),
    (dict(opt=_option(device_error=0x1002)), -3), (dict(opt=_option(k_scale=0x1001)), -3)])
def test_refusals_of_the_cache(L, change, status):
    a = _args(True)
    a.update(change)
    assert _call(L, a) == status


def test_head_sizes(L):
    for D_, status in ((96, -7), (32, -7), (512, -7)):
        a = dict(q_out=_t([T, HQ, D_], B16, 0x100000), q=_t([T, HQ, D_], B16, 0x200000), k_out=None, key=None,
                 positions=None, frequencies=None, q_weight=None, k_weight=None, opt=None)
        assert _call(L, a) == status


@pytest.mark.parametrize("cached", [False, True])
def test_nothing_to_do(L, cached):
    """No rows: a no-op that returns before it touches the device (positions and slots may then be null)."""
    a = _args(cached)
    for k, t in a.items():
        if isinstance(t, pa.PaTensor) and k in ("q_out", "q", "key", "k_out", "value", "positions", "slots"):
            t.shape[0] = 0
            t.data = 0
    assert _call(L, a) == 0


def test_option_struct_layout_matches_the_header(tmp_path):
    import os
    import subprocess
    src = tmp_path / "offsets.c"
    fields = [f for f, _ in pa.PaRotaryOptions._fields_]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pa.h"\nint main(void) { printf("%zu", sizeof(pa_rotary_options));\n'
                   + "".join('printf(" %%zu", offsetof(pa_rotary_options, %s));\n' % f for f in fields) + "return 0; }\n")
    exe = tmp_path / "offsets"
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.check_call(["gcc", "-I", inc, "-o", str(exe), str(src)])
    got = list(map(int, subprocess.check_output([str(exe)]).split()))
    assert got == [ctypes.sizeof(pa.PaRotaryOptions)] + [getattr(pa.PaRotaryOptions, f).offset for f in fields]
    assert len(pa._ROTARY_OPTIONS.pack(1, 2.0, 3.0, 0, 0, 0, 0)) == ctypes.sizeof(pa.PaRotaryOptions)


@pytest.mark.parametrize("cached", [False, True])
@pytest.mark.parametrize("what,by,status", [
    ("q_out", HQ * D * 2, -1), ("q_out", -HQ * D * 2, -1),        # a token on, or back
    ("q_out", D * 2, -1), ("q_out", -D * 2, -1), ("q_out", 16, -1),  # a head on or back, or inside a row
    ("q_out", 3 * HQ * D * 2 + 32, -1), ("q_out", -(T - 1) * HQ * D * 2, -1)])
def test_outputs_that_overlap_their_input(L, cached, what, by, status):
    a = _args(cached)
    a["q_out"].data = a["q"].data + by
    assert _call(L, a) == status


def test_views_of_one_buffer_do_not_overlap():
    """The check itself over every pair of views of one buffer, against the rows' own bytes."""
    import itertools

    def shared(x, y):  # (start, strides, heads) in elements; as rows_shared in pa_validate.h
        rows = lambda v: {(v[0] + t * v[1] + h * v[2] + d) for t in range(3) for h in range(v[3]) for d in range(16)}  # noqa: E731
        return bool(rows(x) & rows(y))

    def check(x, y):
        ts, hs, row, away = x[1], x[2], 16, y[0] - x[0]
        trunc = lambda p, q: int(p / q) if q else 0  # noqa: E731
        for i in (-1, 0, 1):
            t = trunc(away, ts) + i if ts else 0
            left = away - t * ts
            if t >= 3 or -t >= 3:
                continue
            for j in (-1, 0, 1):
                h = trunc(left, hs) + j if hs else 0
                apart = left - h * hs
                if h < x[3] and -h < y[3] and -row < apart < row:
                    return True
        return False

    for ts, hs in ((96, 16), (96, 32), (200, 48), (64, 16)):
        heads = [n for n in (1, 2, 3) if (n - 1) * hs + 16 <= ts]
        for hx, hy in itertools.product(heads, heads):
            for off in range(-3 * ts - 20, 3 * ts + 20, 4):
                x, y = (1000, ts, hs, hx), (1000 + off, ts, hs, hy)
                assert check(x, y) == shared(x, y), (x, y)


def test_refused_side_by_side_outputs(L):
    a = _args(False)
    a["k_out"] = _t([T, HKV, D], B16, a["q"].data + D * 2, strides=[HQ * D, D, 1])
    assert _call(L, a) == -1                  # keys' output over queries
    a = _args(False)
    a["k_out"] = _t([T, HKV, D], B16, a["q_out"].data, strides=[HQ * D, D, 1])
    assert _call(L, a) == -1                  # both outputs in one place
