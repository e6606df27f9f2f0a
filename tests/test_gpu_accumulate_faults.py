"""pa_decode_accumulate where a head has no softmax sum and where a sequence sets an error: nothing is
added, whatever the scores, and whatever the workspace held before the call.  Bounds as
test_gpu_accumulate.py."""
import math

import numpy as np
import pytest
import torch

from test_gpu_accumulate import LENS, _args, _case, _kw

import paged_decode_attention_reshape_gb300 as pa

pytestmark = pytest.mark.gpu

KINDS = [("bf16", 8, 2, 64), ("f16", 12, 2, 128), ("e4m3", 8, 2, 128), ("f32", 6, 2, 64), ("fp4", 8, 2, 128),
         ("fp4", 18, 2, 64)]
IDS = ["%s-%d-%d-%d" % k for k in KINDS]
PARTS = [-1, 64, 0, pa.PA_PARTITION_BALANCED]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    pa.lib()
    torch.cuda.set_device(0)


def spoil(kind, c, g, K, s, head, token, value):
    """Key `token` of (s, head) gets `value` in element 5 (4-bit: NaN in the first group's scale)."""
    blk, off = int(g.block_table[s, token // 16]), token % 16
    if kind == "fp4":
        g.k_cache[blk, head, 8 * c.D + off * (c.D // 16)] = 0x7F
        K[s][token, head, :16] = np.nan
    elif kind == "e4m3":
        g.k_cache[blk, head, off, 5] = 0x7F
        K[s][token, head, 5] = np.nan
    else:
        g.k_cache[blk, head, off, 5] = value
        K[s][token, head, 5] = value


def expected(c, K, q, before):
    """fp64 weights after one call on `before`, and their bounds: a head whose softmax sum is no positive
    number adds nothing."""
    want, tol = before.astype(np.float64), np.zeros(before.shape)
    G = c.Hq // c.Hkv
    for s, L in enumerate(c.lens):
        for h in range(c.Hq if L else 0):
            k = K[s][:, h // G]
            with np.errstate(invalid="ignore"):
                x, B = k @ q[s, h] * c.scale, np.abs(k) @ np.abs(q[s, h]) * c.scale
                p = np.exp(x - x.max())
            if not p.sum() > 0:
                continue
            p /= p.sum()
            B = B[np.isfinite(B)].max()
            e = (c.D / 16 + 4) * 2.0 ** -22 * B
            want[s, h // G, :L] += p
            tol[s, h // G, :L] += p * (2 * e + (L / 16 + 32) * 2.0 ** -24 + (1.45 * B + math.log2(L) + 8) * 2.0 ** -24
                                       + 2.0 ** -22 + G * 2.0 ** -24) + 2.0 ** -120
    tol += 2.0 ** -24 * np.abs(want)
    return want, tol


def poisoned(c, word):
    """A caller's workspace whose arrival counters are zero and whose other words are `word`."""
    ws = torch.full((1 << 24,), word, dtype=torch.int32, device="cuda")
    ws[:(c.S * c.Hkv * -(-(c.Hq // c.Hkv) // 8) * 4 + 255) // 256 * 64] = 0
    return ws


NAN, INF = -1, 0x7F800000


@pytest.mark.parametrize("kind,Hq,Hkv,D", KINDS, ids=IDS)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_heads_without_a_sum_add_nothing(kind, Hq, Hkv, D, value):
    c, g, K = _case(kind, Hq, Hkv, D)
    q = c.q.double().numpy()
    spoil(kind, c, g, K, 4, 1, 333, value)
    spoil(kind, c, g, K, 5, 0, 900, value)
    spoil(kind, c, g, K, 1, 1, 0, value)
    g.q[2, 1, 3] = float("nan")
    q[2, 1, 3] = np.nan
    W = g.block_table.shape[1] * 16
    before = np.exp(np.random.RandomState(2).randn(c.S, Hkv, W)).astype(np.float32)
    want, tol = expected(c, K, q, before)
    for P in PARTS:
        weights = torch.from_numpy(before).cuda()
        pa.pa_decode_accumulate(*_args(c, g), weights, partition_size=P, device_error=g.err, **_kw(kind, g))
        assert pa.pa_check_device_error(g.err) == (0, 0)
        got = weights.double().cpu().numpy()
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (P, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("kind,Hq,Hkv,D", KINDS, ids=IDS)
@pytest.mark.parametrize("word", [NAN, INF], ids=["nan", "inf"])
def test_faults_add_nothing_whatever_the_workspace_held(kind, Hq, Hkv, D, word):
    c, g, K = _case(kind, Hq, Hkv, D)
    W = g.block_table.shape[1] * 16
    before = np.exp(np.random.RandomState(3).randn(c.S, Hkv, W)).astype(np.float32)
    want, tol = expected(c, K, c.q.double().numpy(), before)
    g.block_table[4, 5] = -3
    g.block_table[2, 0] = c.NB
    g.seq_lens[3] = W + 1
    bad_seqs, good = [2, 3, 4], [0, 1, 5]
    for P in PARTS:
        weights = torch.from_numpy(before).cuda()
        pa.pa_decode_accumulate(*_args(c, g), weights, partition_size=P, workspace=poisoned(c, word),
                                device_error=g.err, **_kw(kind, g))
        assert pa.pa_check_device_error(g.err) == (-6, pa.PA_DEVERR_BLOCK_RANGE | pa.PA_DEVERR_SEQLEN_RANGE)
        got = weights.double().cpu().numpy()
        assert np.array_equal(got[bad_seqs], before[bad_seqs].astype(np.float64)), P
        assert (np.abs(got - want) <= tol)[good].all()


@pytest.mark.parametrize("kind,D", [("bf16", 64), ("e4m3", 128)])
@pytest.mark.parametrize("word", [NAN, INF], ids=["nan", "inf"])
def test_timed_out_waits_add_nothing_whatever_the_workspace_held(kind, D, word):
    c, g, _ = _case(kind, 8, 2, D)
    W = g.block_table.shape[1] * 16
    before = np.exp(np.random.RandomState(4).randn(c.S, 2, W)).astype(np.float32)
    for P in PARTS:
        weights = torch.from_numpy(before).cuda()
        pa.pa_decode_accumulate(*_args(c, g), weights, partition_size=P, workspace=poisoned(c, word),
                                device_error=g.err, first_wait_limit=-1, **_kw(kind, g))
        assert pa.pa_check_device_error(g.err) == (-8, pa.PA_DEVERR_WAIT_TIMEOUT)
        assert np.array_equal(weights.cpu().numpy(), before), P
