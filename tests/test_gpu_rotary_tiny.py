"""Norms without an eps over rows whose elements lie below their type's normal numbers."""
import pytest
import torch

import paged_decode_attention_reshape_gb300 as pa
import rotary_model as model

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_norm_of_tiny_rows(dtype, D, interleaved):
    """Elements down to the smallest number of the type, alone and beside zeros and ordinary rows: powers of two
    scale them exactly, so the bound is the one of any other row."""
    least = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    g = torch.Generator().manual_seed(D)
    sizes = [n for n in (least, 3 * least, 40 * least, 1000 * least, 2.0 ** 20 * least, 2.0 ** -52, 2.0 ** -48, 2.0 ** -44, 1.0)
             if n >= least]
    x = torch.zeros(len(sizes) + 1, 3, D, dtype=torch.float64)
    for i, size in enumerate(sizes):
        x[i] = (torch.randn(3, D, generator=g, dtype=torch.float64) * size / least).round() * least
        x[i, 0, 0] = size  # (a row is never all zeros)
        x[i, 1, 1:] = 0.0
        x[i, 1, 0] = -size
        x[i, 2, D - 1] = size
    x[-1] = least  # every element the smallest
    q = x.to(dtype).to(DEV)
    assert bool((q != 0).any(-1).all())
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(dtype).to(DEV)
    f = pa.pa_rotary_frequencies(D).to(DEV)
    pos = torch.arange(len(x), device=DEV) * 37
    for eps in (0.0, 1e-42):
        out = torch.empty_like(q)
        pa.pa_rotary(out, q, None, None, pos, f, w, eps=eps, interleaved=interleaved)
        eps32 = torch.tensor(eps, dtype=torch.float32).double().item()  # (the option's own type)
        model.assert_rows(out, *model.rows(q, pos, f, interleaved, weight=w, eps=eps32), "eps %g" % eps)
