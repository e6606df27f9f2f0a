"""Positions, cache and windows together, as a serving loop uses them: prompts and then single tokens go through
pa_rotary_and_cache and the windowed attention, blocks that leave the window are given back and taken by
other sequences, and every output is checked against fp64 over the rows as they were first written."""
import numpy as np
import pytest
import torch

import paged_decode_attention_reshape_gb300 as pa
import rotary_model as model
import window_cases as wc

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Pool:
    """Free blocks, each handed out poisoned (as a freed block may hold anything)."""

    def __init__(self, n, k_cache, v_cache):
        self.free, self.caches = list(range(n)), (k_cache, v_cache)

    def take(self):
        b = self.free.pop(0)
        for c in self.caches:
            c[b].view(torch.uint8).fill_(0xFF)
        return b

    def give(self, b):
        self.free.append(b)


@pytest.mark.parametrize("kind,dtype,Hq,Hkv,D,R,interleaved,W,K", [
    ("same", torch.bfloat16, 8, 2, 128, 128, False, 70, 4), ("same", torch.float16, 4, 4, 64, 32, True, 33, 0),
    ("e4m3", torch.bfloat16, 16, 2, 128, 64, False, 48, 20), ("fp4", torch.bfloat16, 8, 2, 128, 128, True, 64, 4),
    ("same", torch.float32, 4, 1, 64, 64, False, 40, 3)])
def test_generation(kind, dtype, Hq, Hkv, D, R, interleaved, W, K):
    rng = np.random.RandomState(3)
    S, steps = 4, 40
    prompts = [150, 1, 37, 90]
    eps, scale = 1e-5, D ** -0.5
    width = (max(prompts) + 2 * steps + 15) // 16
    NB = sum((min(n, W) + K) // 16 + 4 for n in prompts) + S * 6
    mode = {"same": pa.PA_KV_AUTO, "e4m3": pa.PA_KV_FP8_E4M3, "fp4": pa.PA_KV_FP4_E2M1}[kind]
    shape = (NB, Hkv, 9 * D) if kind == "fp4" else (NB, Hkv, 16, D)
    kc, vc = [torch.zeros(shape, dtype=dtype if kind == "same" else torch.uint8, device=DEV) for _ in range(2)]
    kv_scale = None if kind == "same" else torch.full((1,), 0.05 if kind == "e4m3" else 1.0, device=DEV)
    kv = dict(k_scale=kv_scale, v_scale=kv_scale)
    pool = Pool(NB, kc, vc)
    freq = pa.pa_rotary_frequencies(R, 10000.0, pa.PA_ROTARY_PARTS, 4.0, 64.0).to(DEV)
    wq, wk = [torch.from_numpy((1 + 0.2 * rng.randn(D)).astype(np.float32)).to(dtype).to(DEV) for _ in range(2)]
    rot = dict(eps=eps, interleaved=interleaved, magnitude=1.0 + 0.1 * np.log(4.0))
    table = torch.full((S, width), -1, dtype=torch.int32)
    lens = [0] * S
    hist = [[np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))] for _ in range(S)]  # cached values, kept on the host
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    reused = 0

    def step(news):
        nonlocal reused
        n = sum(news)
        slots, pos = [], []
        for s, m in enumerate(news):
            for p in range(lens[s], lens[s] + m):
                if table[s, p // 16] < 0:
                    table[s, p // 16] = pool.take()
                slots.append(int(table[s, p // 16]) * 16 + p % 16)
                pos.append(p)
            lens[s] += m
        x = torch.from_numpy(rng.randn(n, Hq + 2 * Hkv, D).astype(np.float32)).to(dtype).to(DEV)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        slots, pos = torch.tensor(slots, device=DEV), torch.tensor(pos, device=DEV)
        want_q = model.rows(q, pos, freq, interleaved, rot["magnitude"], wq, eps)
        pa.pa_rotary_and_cache(q, q, k, v, kc, vc, pos, slots, freq, mode, wq, wk, device_error=err, **rot, **kv)
        model.assert_rows(q, *want_q)  # (in place)
        back = dtype if kind == "same" else torch.float32
        kb, vb = [torch.empty(n, Hkv, D, dtype=back, device=DEV) for _ in range(2)]
        pa.pa_gather_cache(kb, vb, kc, vc, slots, **kv)
        if kind == "same":
            model.assert_rows(kb, *model.rows(k, pos, freq, interleaved, rot["magnitude"], wk, eps))
            assert torch.equal(vb, v)
        at = 0
        for s, m in enumerate(news):
            for i, b in enumerate((kb, vb)):
                hist[s][i] = np.concatenate([hist[s][i], b[at:at + m].double().cpu().numpy()])
            at += m
        out = torch.full((n, Hq, D), float("nan"), dtype=dtype, device=DEV)
        bt, sl = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
        if all(m == 1 for m in news):
            pa.pa_decode_window(out, q.contiguous(), kc, vc, bt, sl, scale, Hkv, W, K, device_error=err, **kv)
        else:
            starts = torch.from_numpy(np.concatenate([[0], np.cumsum(news)]).astype(np.int32)).to(DEV)
            pa.pa_attention_window(out, q.contiguous(), kc, vc, starts, bt, sl, scale, Hkv, max(news), W, K, device_error=err, **kv)
        assert pa.pa_check_device_error(err) == (0, 0)
        c = wc.Case()
        c.q, c.dtype, c.lens, c.nq, c.Hkv, c.Hq, c.D, c.W, c.K = q.cpu(), dtype, lens, list(news), Hkv, Hq, D, W, K
        c.scale, c.alibi, c.vals = scale, None, [[h[0] for h in hist], [h[1] for h in hist]]
        ref, tol = wc.reference(c)
        wc.check(out, (ref, tol), "lengths %s" % lens)
        # blocks without a token that any later query sees go back
        for s in range(S):
            for b in range(K // 16 + (K % 16 > 0), max(0, lens[s] + 1 - W) // 16):
                if table[s, b] >= 0:
                    pool.give(int(table[s, b]))
                    table[s, b] = -1
                    reused += 1

    step(prompts)
    for i in range(steps):
        step([1] * S if i % 7 else [3, 1, 2, 5])
    assert reused >= 8


def test_keys_moved_to_new_positions():
    """Keys of a cached sequence rotated from the positions they were written at to others (their places after
    an eviction), by pa_gather_cache, pa_rotary over the differences and the write: the rows of a fresh write."""
    T, Hkv, D = 50, 2, 128
    g = torch.Generator().manual_seed(5)
    k = torch.randn(T, Hkv, D, generator=g).to(DEV)
    f = pa.pa_rotary_frequencies(D).to(DEV)
    old, new = torch.arange(T, device=DEV) * 3 + 1000, torch.arange(T, device=DEV)
    kc, vc = [torch.zeros(4, Hkv, 16, D, device=DEV) for _ in range(2)]
    slots = torch.arange(T, device=DEV)
    pa.pa_rotary_and_cache(None, None, k, k, kc, vc, old, slots, f)
    rows, vals = torch.empty_like(k), torch.empty_like(k)
    pa.pa_gather_cache(rows, vals, kc, vc, slots)
    pa.pa_rotary_and_cache(None, None, rows, vals, kc, vc, new - old, slots, f)
    pa.pa_gather_cache(rows, vals, kc, vc, slots)
    want, bound = model.rows(k, new, f)
    # two rotations, each off by 6 u (|a| + |b|) <= 6 sqrt(2) u of the pair's length, which rotations keep
    pair = torch.hypot(k[..., :64], k[..., 64:]).repeat(1, 1, 2).double().cpu()
    assert bool(((rows.double().cpu() - want).abs() <= 18 * 2.0 ** -24 * pair).all())
    assert torch.equal(vals, k)
