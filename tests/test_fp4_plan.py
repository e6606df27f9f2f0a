"""The plan of a decode over 4-bit pages, on the host."""
import pytest

import paged_decode_attention_reshape_gb300 as pa

SM = 152


@pytest.mark.parametrize("S,MB", [(511, 1 << 23), (32, 1 << 26), (256, 1 << 23)])
def test_tables_past_32_bits_of_pages_are_not_balanced(S, MB):
    """The balanced splits number the pages of all sequences in 32 bits: with more entries than
    that (a broadcast table has them in little memory) the plan is another, and asking is refused."""
    assert S * MB > 2**31 - 1
    assert pa.pa_decode_plan(S, 32, 8, 128, MB, pa.PA_FP4_E2M1, sm_count=SM)[0] != pa.PA_PARTITION_BALANCED
    with pytest.raises(pa.PAError) as e:
        pa.pa_decode_plan(S, 32, 8, 128, MB, pa.PA_FP4_E2M1, sm_count=SM, partition_size=pa.PA_PARTITION_BALANCED)
    assert pa.STATUS[e.value.status] == "PA_ERR_UNSUPPORTED_SHAPE"


@pytest.mark.parametrize("S,MB", [(511, (2**31 - 1) // 511), (256, 256)])
def test_tables_within_32_bits_stay_balanced(S, MB):
    plan = pa.pa_decode_plan(S, 32, 8, 128, MB, pa.PA_FP4_E2M1, sm_count=SM)
    assert plan[0] == pa.PA_PARTITION_BALANCED


def test_tables_of_more_than_2_to_26_blocks_are_refused():
    """Lengths are rounded up to stages of 64 tokens in 32 bits (host checks only, nothing is launched)."""
    import ctypes

    from test_abi import _t

    H, D, MB = 2, 128, (1 << 26) + 1
    q = _t([1, 2 * H, D], pa.PA_BF16)
    page = _t([4, H, 9 * D], pa.PA_FP4_E2M1)
    table = _t([1, MB], pa.PA_I32)
    args = [ctypes.byref(x) for x in (_t([1, 2 * H, D], pa.PA_BF16), q, page, page, table, _t([1], pa.PA_I32))]
    assert pa.lib().pa_decode_opt(*args, 1.0, H, None, None) == -7
