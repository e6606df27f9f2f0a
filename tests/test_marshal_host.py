"""The binding's two ways to describe tensors, in Python and natively (csrc/pa_marshal.cpp), agree byte
for byte and refuse alike."""
import pytest
import torch

import paged_decode_attention_reshape_gb300 as pa


@pytest.fixture(scope="module")
def native():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    return pytest.importorskip("paged_decode_attention_reshape_gb300._marshal").describe


def tensors():
    x = torch.zeros(6, 10, 16, 64)
    yield from (x, x[1:, 2:5], x.permute(0, 2, 1, 3), x[:, :, 3], x[0, 0, 0], x[:0], x[2:2], x[0, 0, 0, 0], x[:1].expand(5, 10, 16, 64))
    for dt in (torch.float32, torch.bfloat16, torch.float16, torch.uint8, torch.float8_e4m3fn, torch.int32, torch.int64):
        yield torch.zeros(3, 4, 9 * 64, dtype=dt)
        yield torch.zeros(7, dtype=dt)[::2]
    yield torch.zeros(2, 3, 16, 128, dtype=torch.uint8)
    yield torch.nn.Parameter(torch.zeros(2, 2))


def test_same_bytes(native):
    for t in tensors():
        assert native(b"t", t) == (pa._desc(t),)
        assert native(b"c", t) == (pa._cache(t),)
    a, b = torch.zeros(2, 3, 4, dtype=torch.uint8), torch.zeros(5)
    assert native(b"cttt", a, None, b, a) == (pa._cache(a), None, pa._desc(b), pa._desc(a))
    assert native(b"") == ()


def test_refusals(native):
    for dt in (torch.float64, torch.bool, torch.complex64):
        for f in (lambda t: native(b"t", t), pa._desc):
            with pytest.raises(KeyError):
                f(torch.zeros(2, dtype=dt))
    for f in (lambda t: native(b"t", t), pa._desc):
        with pytest.raises(ValueError):
            f(torch.zeros(1, 1, 1, 1, 1, 1))
    for bad in (3, "x", [1], object()):
        with pytest.raises(TypeError):
            native(b"t", bad)
    for args in ((), (b"tt", torch.zeros(1)), ("t", torch.zeros(1))):
        with pytest.raises(TypeError):
            native(*args)


def test_for_this_torch(native):
    from paged_decode_attention_reshape_gb300 import _marshal
    assert _marshal.torch == torch.__version__
    pa.lib()
    assert pa._describe is native
