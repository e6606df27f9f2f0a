"""Attention cases under a window, built on the host, and their fp64 reference with the error bound that
the tests hold outputs to.

Everything that no query of its sequence sees is poison: such tokens hold NaN, the table entries of
blocks without a seen token are out of range or name other sequences' blocks, and so is the padding.

Bound of one output element, with p and A = sum_t p_t |v_t| in fp64 over the n tokens seen:
  half a step of the output's type, relative to the value (f16: 2^-25 absolute below its normal range);
  A (2 e + 2^-16 + n 2^-23): e bounds the error of a logit: D / 16 tensor-core sums, each off by at most
  2^-22 of the sum of magnitudes B = scale sum_d |q_d k_d| (with ALiBi, B counts the bias), and four fp32
  roundings, e = (D / 16 + 4) 2^-22 max B (the fp32 kernel sums D / 32 products and five levels of lanes,
  less than that); 2^-16 covers 2^x and p in two halves of its 16-bit type (bf16: 2^-18); n 2^-23 the fp32
  sums over tokens, one rounding and one rescale each;
  2^-25 sum_t |v_t|: the f16 halves of a p below 2^-14 (p counts from a maximum never above the true
  one, so the sum that divides is at least 1)."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle

HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}


class Case:
    pass


def sees(t, P, W, K):
    return (t <= P) & ((t > P - W) | (t < K))


def make(lens, Hq, Hkv, D, W, K, dtype=torch.bfloat16, cache="same", nq=None, seed=0, alibi=None, nhd=False,
         k_scale=1.0, v_scale=1.0, extra_rows=0, sigma=1.0) -> Case:
    """cache: "same" (dtype's), "e4m3" or "fp4".  nq: new tokens per sequence (None: pa_decode_window)."""
    rng = np.random.RandomState(seed)
    c = Case()
    c.S, c.Hq, c.Hkv, c.D, c.W, c.K, c.lens, c.dtype, c.nq = len(lens), Hq, Hkv, D, W, K, list(lens), dtype, nq
    c.cache, c.scale = cache, 1.0 / math.sqrt(D)
    c.alibi = None if alibi is None else np.asarray(alibi, np.float32)
    c.k_scale, c.v_scale = np.asarray(k_scale, np.float32), np.asarray(v_scale, np.float32)
    assert c.k_scale.ndim == c.v_scale.ndim  # (one stride for both)
    news = [1] * c.S if nq is None else nq
    shown = []  # per sequence: which tokens some query sees
    for L, n in zip(lens, news):
        t = np.arange(L)
        shown.append((t < K) | (t > L - max(n, 1) - W) if L else np.zeros(0, bool))
    blocks = [sorted({int(t) // 16 for t in np.flatnonzero(m)}) for m in shown]
    c.width = max([(L + 15) // 16 for L in lens] + [1]) + 2
    c.NB = sum(map(len, blocks)) + 3
    order = rng.permutation(c.NB)
    c.table = rng.choice(np.array([-1, -2 ** 31, c.NB, 2 ** 31 - 1], dtype=np.int64), size=(c.S, c.width)).astype(np.int32)
    at = 0
    for s, bs in enumerate(blocks):
        c.table[s, bs] = order[at:at + len(bs)]
        at += len(bs)
    if cache == "fp4":
        pool = np.full((2, c.NB, Hkv, 9 * D), 0xFF, np.uint8)
    else:
        shape = (2, c.NB, 16, Hkv, D) if nhd else (2, c.NB, Hkv, 16, D)
        pool = torch.empty(shape, dtype=torch.uint8 if cache == "e4m3" else dtype)
        pool.view(torch.uint8).fill_(0xFF)
        if nhd:
            pool = pool.permute(0, 1, 3, 2, 4)
    c.vals = [[], []]
    for s, L in enumerate(lens):
        t = np.flatnonzero(shown[s])
        blk, off = c.table[s][t // 16].astype(np.int64), t % 16
        for i, sc in enumerate((c.k_scale, c.v_scale)):
            x = (rng.randn(len(t), Hkv, D) * sigma).astype(np.float32)
            full = np.full((L, Hkv, D), np.nan)
            if cache == "fp4":
                code, sg = oracle.fp4_quantize(x, sc)
                oracle.fp4_store(pool[i], blk * 16 + off, code, sg)
                full[t] = oracle.fp4_values(code, sg, sc)
            elif cache == "e4m3":
                code = torch.from_numpy(x / 0.05).clamp(-448, 448).to(torch.float8_e4m3fn)
                pool[i][blk, :, off] = code.view(torch.uint8)
                full[t] = code.to(torch.float64).numpy() * (sc.reshape(-1, 1) if sc.ndim else sc).astype(np.float64)
            else:
                v = torch.from_numpy(x).to(dtype)
                pool[i][blk, :, off] = v
                full[t] = v.double().numpy()
            c.vals[i].append(full)
    c.pool = pool
    rows = c.S if nq is None else sum(nq)
    c.q = torch.from_numpy(rng.randn(rows + extra_rows, Hq, D).astype(np.float32)).to(dtype)
    return c


def on_gpu(c):
    g = Case()
    if c.cache == "fp4":
        g.k_cache, g.v_cache = torch.from_numpy(c.pool[0]).cuda(), torch.from_numpy(c.pool[1]).cuda()
    else:
        pool = c.pool.cuda()  # (keeps the layout)
        g.k_cache, g.v_cache = pool[0], pool[1]
    g.q = c.q.cuda()
    g.out = torch.full_like(g.q, float("nan"))
    g.block_table = torch.from_numpy(c.table).cuda()
    g.seq_lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    quantised = c.cache != "same"
    g.k_scale = torch.from_numpy(np.atleast_1d(c.k_scale)).cuda() if quantised else None
    g.v_scale = torch.from_numpy(np.atleast_1d(c.v_scale)).cuda() if quantised else None
    g.stride = 0 if c.k_scale.ndim == 0 else 1
    g.alibi = None if c.alibi is None else torch.from_numpy(c.alibi).cuda()
    g.err = torch.zeros(1, dtype=torch.int32, device="cuda")
    g.ws = torch.zeros(320 << 20, dtype=torch.uint8, device="cuda")
    if c.nq is not None:
        g.starts = torch.from_numpy(np.concatenate([[0], np.cumsum(c.nq)]).astype(np.int32)).cuda()
    return g


def run(c, g, partition_size=0, ws=True, nq_max=None, **kw):
    import paged_decode_attention_reshape_gb300 as pa
    g.out.fill_(float("nan"))
    opt = dict(k_scale=g.k_scale, v_scale=g.v_scale, scale_stride=g.stride, alibi_slopes=g.alibi,
               partition_size=partition_size, workspace=g.ws if ws else None, device_error=g.err, **kw)
    if c.nq is None:
        pa.pa_decode_window(g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, c.Hkv, c.W, c.K, **opt)
    else:
        pa.pa_attention_window(g.out, g.q, g.k_cache, g.v_cache, g.starts, g.block_table, g.seq_lens, c.scale, c.Hkv,
                               nq_max or max(c.nq + [1]), c.W, c.K, **opt)
    return g.out


def reference(c):
    """(outputs fp64, their bounds)."""
    q = c.q.double().numpy()
    out, tol = np.zeros_like(q), np.zeros_like(q)
    row, G = 0, c.Hq // c.Hkv
    for s, L in enumerate(c.lens):
        n = 1 if c.nq is None else c.nq[s]
        for i in range(n):
            P = L - n + i
            if P >= 0:
                t = np.flatnonzero(sees(np.arange(L), P, c.W, c.K))
                for g in range(c.Hkv):
                    k, v = c.vals[0][s][t, g], c.vals[1][s][t, g]
                    qs = q[row + i, g * G:(g + 1) * G]
                    x, B = qs @ k.T * c.scale, np.abs(qs) @ np.abs(k).T * c.scale
                    if c.alibi is not None:
                        bias = c.alibi[g * G:(g + 1) * G, None].astype(np.float64) * (t - P)
                        x, B = x + bias, B + np.abs(bias)
                    p = np.exp(x - x.max(-1, keepdims=True))
                    p /= p.sum(-1, keepdims=True)
                    out[row + i, g * G:(g + 1) * G] = p @ v
                    e = (c.D / 16 + 4) * 2.0 ** -22 * B.max(-1, keepdims=True)
                    tol[row + i, g * G:(g + 1) * G] = (p @ np.abs(v)) * (2 * e + 2.0 ** -16 + len(t) * 2.0 ** -23) \
                        + 2.0 ** -25 * np.abs(v).sum(0)
        row += n
    tol += HALF[c.dtype] * (np.abs(out) + tol) + (2.0 ** -25 if c.dtype == torch.float16 else 0)
    return out, tol


def check(got, want, what=""):
    ref, tol = want
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d outside their bounds, worst %.3g of it, first %s" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - ref) / tol), np.argwhere(bad)[:3].tolist())
