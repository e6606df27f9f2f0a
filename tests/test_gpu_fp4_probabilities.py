"""How finely the attention over a 4-bit cache holds its softmax weights, with either query type.

Every value of V is +c or -c and, per output element, as many are one as the other; the logits are
within 2^-7 or so of each other.  So the weights are nearly equal, the output is the small rest of
large terms that cancel, and rounding it to its type is no longer what bounds its error: an output
element is off by at most (fp4_cases.py's terms, p in two halves whatever the query's type)
  half a step of the output type, relative to the value, plus A (2 e + 2^-17) + 2^-25 sum_t |v_t|,
  A = sum_t p_t |v_t| = c.
Weights held in 11 bits are off by up to 2^-12 of themselves each, 2^-12.8 in the mean of squares, and
n of them with random signs by 2^-12.8 / sqrt(n) of A: 2^-14.8 for 16 tokens, where the bound's terms
are about 2^-16."""
import numpy as np
import pytest
import torch

import fp4_cases
import oracle

import paged_decode_attention_reshape_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    pa.lib()
    torch.cuda.set_device(0)


def near_equal_weights(S, Hq, Hkv, D, lens, dtype, nq=None):
    """fp4_cases.make, with V balanced and the query made small."""
    c = fp4_cases.make(S, Hq, Hkv, D, lens, dtype, seed=D + Hq, nq=nq)
    rng = np.random.default_rng(D)
    for s, L in enumerate(lens):
        half = np.where(np.arange(L) < L // 2, 1.0, -1.0).astype(np.float32)
        x = rng.permuted(np.broadcast_to(half[:, None, None], (L, Hkv, D)), axis=0)
        code, sg = oracle.fp4_quantize(x, c.v_scale)
        slots = c.table[s][np.arange(L) // 16].astype(np.int64) * 16 + np.arange(L) % 16
        oracle.fp4_store(c.pool[1], slots, code, sg)
        c.V[s] = oracle.fp4_values(code, sg, c.v_scale)
        assert (c.V[s].sum(0) == 0).all()
    c.q = (c.q.float() * 2.0 ** -8).to(dtype)
    return c


def bounds(c):
    """(outputs fp64, bounds), p in two halves."""
    ref, tol, probs = fp4_cases.reference(c)
    if c.dtype == torch.bfloat16:      # fp4_cases.py allows p 11 bits here
        row = 0
        for s, L in enumerate(c.lens):
            for i in range(1 if c.nq is None else c.nq[s]):
                for h in range(c.Hq):
                    p = probs[s][i, h]
                    tol[row, h] -= 2.0 ** -11 * (p @ np.abs(c.V[s][:, h // (c.Hq // c.Hkv)]))
                row += 1
    return ref, tol


LENS = [16, 30, 64, 128]


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (32, 8, 128), (8, 1, 128), (6, 2, 256)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_decode(Hq, Hkv, D, dt):
    c = near_equal_weights(len(LENS), Hq, Hkv, D, LENS, dt)
    ref, tol = bounds(c)
    g = fp4_cases.to_gpu(c)
    for P in (-1, 16, -2, pa.PA_PARTITION_BALANCED):
        g.out.fill_(float("nan"))
        pa.pa_decode_opt(g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, Hkv,
                         partition_size=P, workspace=g.ws, device_error=g.err)
        assert pa.pa_check_device_error(g.err) == (0, 0)
        fp4_cases.check(g.out, ref, tol, "partition %d" % P)
        g.ws.zero_()


def test_varlen():
    c = near_equal_weights(4, 8, 2, 128, LENS, torch.bfloat16, nq=[1, 1, 1, 1])
    ref, tol = bounds(c)
    g = fp4_cases.to_gpu(c)
    pa.pa_attention_varlen(g.out, g.q, g.k_cache, g.v_cache, g.starts, g.block_table, g.seq_lens, c.scale, 2, 3,
                           device_error=g.err)
    assert pa.pa_check_device_error(g.err) == (0, 0)
    fp4_cases.check(g.out, ref, tol)


def test_many_units():
    """The split over warps."""
    lens = [16 + 2 * (i % 40) for i in range(40)]
    c = near_equal_weights(40, 16, 8, 128, lens, torch.bfloat16)
    ref, tol = bounds(c)
    g = fp4_cases.to_gpu(c)
    pa.pa_decode_opt(g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, 8,
                     partition_size=pa.PA_PARTITION_BALANCED, device_error=g.err)
    assert pa.pa_check_device_error(g.err) == (0, 0)
    fp4_cases.check(g.out, ref, tol)
