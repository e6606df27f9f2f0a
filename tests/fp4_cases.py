"""Attention cases over 4-bit caches, built on the host by the oracle's codec, and their fp64
reference with the error bound the tests hold outputs to.

Bound of one output element, with p and A = sum_t p_t |v_t| in fp64:
  half a step of the output type, relative to the value (bf16 2^-8, f16 2^-11, f16 below its
  normal range 2^-25 absolute), plus A (2 e + 2^-17 + r), where e bounds the error of a logit,
  2^-17 covers the fp32 sums over tokens, the 2^x function and the two halves (22 bits) that p
  is held in for an f16 query, and r = 2^-11 with a bf16 query, for which p is held in one f16:
  half a step of f16, relative.
The codes, their scales and the query (scaled by a power of two, f16) enter the products
exactly; a logit is D / 16 fp32 tensor-core sums, each off by at most 2^-22 of the sum of
magnitudes B = scale sum_d |q_d k_d|, and four fp32 roundings: e = (D / 16 + 4) 2^-22 max B
(with ALiBi, B counts the bias too).
The halves of p are f16, whose step is 2^-24 below its normal range, so a p under 2^-14 is held
to within half of that, 2^-25, and not to 22 bits.  p counts from a running maximum m that is
never above the true one, so the sum of all p that divides them is at least 1: this adds at most
2^-25 sum_t |v_t|."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class Fp4Case:
    pass


def make(S, Hq, Hkv, D, lens, dtype=torch.bfloat16, seed=0, k_scale=1.0, v_scale=1.0, sigma=1.0, nq=None,
         alibi=None, interleaved=False) -> Fp4Case:
    """nq: new query tokens per sequence (None: one each, pa_decode).  Bytes that hold no token are
    0xFF: code -6 and scale NaN."""
    rng = np.random.RandomState(seed)
    c = Fp4Case()
    c.S, c.Hq, c.Hkv, c.D, c.lens, c.dtype, c.nq = S, Hq, Hkv, D, list(lens), dtype, nq
    c.scale = 1.0 / math.sqrt(D)
    c.k_scale, c.v_scale = np.asarray(k_scale, np.float32), np.asarray(v_scale, np.float32)
    c.alibi = None if alibi is None else np.asarray(alibi, np.float32)
    need = [(L + 15) // 16 for L in lens]
    c.NB, c.width = sum(need) + 4, max(need + [1]) + 2
    order = rng.permutation(c.NB)
    c.table = np.full((S, c.width), -1, np.int32)
    pool = np.full((2, c.NB, Hkv, 9 * D), 0xFF, np.uint8)
    c.K, c.V = [], []
    at = 0
    for s, L in enumerate(lens):
        c.table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        slots = c.table[s][np.arange(L) // 16].astype(np.int64) * 16 + np.arange(L) % 16
        for i, (vals, sc) in enumerate(((c.K, c.k_scale), (c.V, c.v_scale))):
            x = (rng.randn(L, Hkv, D) * sigma).astype(np.float32)
            code, sg = oracle.fp4_quantize(x, sc)
            oracle.fp4_store(pool[i], slots, code, sg)
            vals.append(oracle.fp4_values(code, sg, sc))
    c.pool = pool
    rows = S if nq is None else sum(nq)
    c.q = torch.from_numpy(rng.randn(rows, Hq, D).astype(np.float32)).to(dtype)
    c.interleaved = interleaved
    return c


def to_gpu(c):
    g = Fp4Case()
    if c.interleaved:
        both = torch.from_numpy(np.ascontiguousarray(c.pool.transpose(1, 0, 2, 3))).cuda()
        g.k_cache, g.v_cache = both[:, 0], both[:, 1]
    else:
        g.k_cache, g.v_cache = torch.from_numpy(c.pool[0]).cuda(), torch.from_numpy(c.pool[1]).cuda()
    g.q = c.q.cuda()
    g.out = torch.full_like(g.q, float("nan"))
    g.block_table = torch.from_numpy(c.table).cuda()
    g.seq_lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    g.k_scale = torch.from_numpy(np.atleast_1d(c.k_scale)).cuda()
    g.v_scale = torch.from_numpy(np.atleast_1d(c.v_scale)).cuda()
    g.stride = 0 if c.k_scale.ndim == 0 else 1
    g.alibi = None if c.alibi is None else torch.from_numpy(c.alibi).cuda()
    g.err = torch.zeros(1, dtype=torch.int32, device="cuda")
    g.ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    if c.nq is not None:
        g.starts = torch.from_numpy(np.concatenate([[0], np.cumsum(c.nq)]).astype(np.int32)).cuda()
    return g


def reference(c):
    """(outputs fp64, their bounds, attention weights [S] of [n, Hq, L])."""
    q = c.q.double().numpy()
    out, tol, probs = np.zeros_like(q), np.zeros_like(q), []
    row = 0
    G = c.Hq // c.Hkv
    for s, L in enumerate(c.lens):
        n = 1 if c.nq is None else c.nq[s]
        pr = np.zeros((n, c.Hq, L))
        for i in range(n):
            see = L - n + i + 1 if c.nq is not None else L
            for h in range(c.Hq):
                if see <= 0:
                    continue
                K, V = c.K[s][:see, h // G], c.V[s][:see, h // G]
                x = K @ q[row + i, h] * c.scale
                B = np.abs(K) @ np.abs(q[row + i, h]) * c.scale
                if c.alibi is not None:
                    bias = c.alibi[h].astype(np.float64) * (np.arange(see) - (see - 1))
                    x, B = x + bias, B + np.abs(bias)
                p = np.exp(x - x.max())
                p /= p.sum()
                pr[i, h, :see] = p
                out[row + i, h] = p @ V
                e = (c.D / 16 + 4) * 2.0 ** -22 * B.max()
                tol[row + i, h] = p @ np.abs(V) * (2 * e + 2.0 ** -17 + (2.0 ** -11 if c.dtype == torch.bfloat16 else 0)) + 2.0 ** -25 * np.abs(V).sum(0)
        probs.append(pr)
        row += n
    tol += HALF[c.dtype] * np.abs(out) + (2.0 ** -25 if c.dtype == torch.float16 else 0)
    return out, tol, probs


def check(got, ref, tol, what=""):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d outside their bounds, worst %.3g over it, first %s" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - ref) - tol), np.argwhere(bad)[:3].tolist())
