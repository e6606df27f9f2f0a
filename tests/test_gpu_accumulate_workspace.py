"""One caller workspace, zero-filled once, for accumulating and plain decodes of one shape, split and
unsplit, in any order."""
import numpy as np
import pytest
import torch

import fp4_cases
from gpu_cases import assert_close, make_case, reference, to_gpu
from test_gpu_accumulate import _args, _kw, expected

import paged_decode_attention_reshape_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    pa.lib()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp4"])
def test_shared_by_split_and_unsplit_calls(kind):
    lens = [300, 1, 129, 640]
    if kind == "fp4":
        c = fp4_cases.make(4, 8, 2, 128, lens, torch.bfloat16, seed=3)
        g, K = fp4_cases.to_gpu(c), c.K
        ref, otol, _ = fp4_cases.reference(c)
    else:
        c = make_case(4, 8, 2, 128, lens, dtype={"bf16": torch.bfloat16, "f32": torch.float32}[kind], seed=3)
        g, K, ref = to_gpu(c), c.Kval, reference(c)
    W = g.block_table.shape[1] * 16
    want, tol = expected(c, K, np.zeros((4, 2, W), np.float32))
    sizes = [pa.pa_decode_accumulate_workspace_size(4, 8, 2, 128, g.block_table.shape[1], P) for P in (-1, 64)]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    assert sizes[0] < sizes[1]
    for accumulate, P, size in ((True, -1, sizes[0]), (True, 64, sizes[1]), (True, -1, sizes[1]), (False, 64, sizes[1]),
                                (True, -1, sizes[0]), (False, 64, sizes[1]), (True, 64, sizes[1]),
                                (False, 64, sizes[1])):
        g.out.fill_(float("nan"))
        weights = torch.zeros(4, 2, W, device="cuda")
        if accumulate:
            pa.pa_decode_accumulate(*_args(c, g), weights, partition_size=P, workspace=ws[:size],
                                    device_error=g.err, **_kw(kind, g))
            assert (np.abs(weights.double().cpu().numpy() - want) <= tol).all(), P
        else:
            pa.pa_decode_opt(*_args(c, g), partition_size=P, workspace=ws, device_error=g.err, **_kw(kind, g))
        assert pa.pa_check_device_error(g.err) == (0, 0)
        if kind == "fp4":
            fp4_cases.check(g.out, ref, otol, "outputs, P %d" % P)
        else:
            assert_close(g.out.double().cpu().numpy(), ref, "outputs, P %d" % P)
