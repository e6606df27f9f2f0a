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


@pytest.mark.parametrize("kind,nhd", [("same", False), ("same", True), ("e4m3", False), ("fp4", False)])
def test_blocks_past_4_gib(kind, nhd):
    """The write and both windowed calls over blocks whose byte offsets pass 2^32."""
    Hkv, Hq, D, W, K, lens = 2, 8, 128, 100, 4, [300, 257, 40]
    per = {"same": Hkv * 16 * D * 2, "e4m3": Hkv * 16 * D, "fp4": Hkv * 9 * D}[kind]
    base = (1 << 32) // per + 77
    need = [(n + 15) // 16 for n in lens]
    NB = base + sum(need) + 5
    if kind == "fp4":
        caches = [torch.empty(NB, Hkv, 9 * D, dtype=torch.uint8, device=DEV) for _ in range(2)]
    else:
        shape = (NB, 16, Hkv, D) if nhd else (NB, Hkv, 16, D)
        caches = [torch.empty(shape, dtype=torch.bfloat16 if kind == "same" else torch.uint8, device=DEV) for _ in range(2)]
        if nhd:
            caches = [c.permute(0, 2, 1, 3) for c in caches]
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)) + base
    table = torch.full((3, max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n].int()
        at += n
    slots = torch.cat([table[s][torch.arange(n) // 16].long() * 16 + torch.arange(n) % 16 for s, n in enumerate(lens)]).to(DEV)
    pos = torch.cat([torch.arange(n) for n in lens]).to(DEV)
    T = sum(lens)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    q, k, v = x[:, :Hq].contiguous(), x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    mode = {"same": pa.PA_KV_AUTO, "e4m3": pa.PA_KV_FP8_E4M3, "fp4": pa.PA_KV_FP4_E2M1}[kind]
    sc = None if kind == "same" else torch.full((1,), 0.05 if kind == "e4m3" else 1.0, device=DEV)
    kv = dict(k_scale=sc, v_scale=sc)
    f = pa.pa_rotary_frequencies(D).to(DEV)
    pa.pa_rotary_and_cache(q, q, k, v, *caches, pos, slots, f, mode, **kv)
    back = torch.bfloat16 if kind == "same" else torch.float32
    kb, vb = [torch.empty(T, Hkv, D, dtype=back, device=DEV) for _ in range(2)]
    pa.pa_gather_cache(kb, vb, *caches, slots, **kv)
    if kind == "same":
        model.assert_rows(kb, *model.rows(k, pos, f))
        assert torch.equal(vb, v)
    ends = np.cumsum(lens)
    c = wc.Case()
    c.dtype, c.lens, c.Hkv, c.Hq, c.D, c.W, c.K, c.scale, c.alibi = torch.bfloat16, lens, Hkv, Hq, D, W, K, D ** -0.5, None
    c.vals = [[y[e - n:e].double().cpu().numpy() for e, n in zip(ends, lens)] for y in (kb, vb)]
    bt, sl = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    for nq in (None, [70, 3, 20]):
        c.nq = nq
        rows = [e - 1 for e in ends] if nq is None else [i for e, n in zip(ends, nq) for i in range(e - n, e)]
        c.q = q[rows].cpu()
        out = torch.full((len(rows), Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        if nq is None:
            pa.pa_decode_window(out, q[rows].contiguous(), *caches, bt, sl, c.scale, Hkv, W, K, **kv)
        else:
            starts = torch.from_numpy(np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)).to(DEV)
            pa.pa_attention_window(out, q[rows].contiguous(), *caches, starts, bt, sl, c.scale, Hkv, max(nq), W, K, **kv)
        wc.check(out, wc.reference(c), "new tokens %s" % nq)


@pytest.mark.parametrize("rows", [0, 3])
def test_rotation_right_before_a_step(rows):
    """Queries rotated in place by a long kernel and read by the step right behind it, which starts early where it
    writes rows and may not where it has none to write."""
    S, Hq, Hkv, D, T = 3, 8, 2, 128, 40000
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(T, Hq, D, device=DEV, generator=gen).to(torch.bfloat16)
    pos = torch.arange(T, device=DEV)
    freq = pa.pa_rotary_frequencies(D).to(DEV)
    kc, vc = [torch.randn(30, Hkv, 16, D, device=DEV, generator=gen).to(torch.bfloat16) for _ in range(2)]
    table = torch.arange(30, dtype=torch.int32, device=DEV).view(3, 10)
    lens = torch.tensor([150, 7, 90], dtype=torch.int32, device=DEV)
    key, value = [torch.randn(rows, Hkv, D, device=DEV, generator=gen).to(torch.bfloat16) for _ in range(2)]
    slots = torch.tensor([149, 160 + 6, 320 + 89], device=DEV)[:rows]
    starts = torch.tensor([0, 1, 2, 3] if rows else [0] * 4, dtype=torch.int32, device=DEV)
    rotated, want, got = x.clone(), torch.empty(S, Hq, D, dtype=x.dtype, device=DEV), torch.empty_like(x[:S])
    ks, vs = kc.clone(), vc.clone()
    pa.pa_rotary(rotated, rotated, None, None, pos, freq)
    torch.cuda.synchronize()
    if rows:
        pa.pa_reshape_and_cache(key, value, ks, vs, slots)
    pa.pa_decode_opt(want, rotated[T - S:], ks, vs, table, lens, D ** -0.5, Hkv, partition_size=-1)
    torch.cuda.synchronize()
    for _ in range(5):
        now = x.clone()
        pa.pa_rotary(now, now, None, None, pos, freq)
        pa.pa_decode_step(got, now[T - S:], key, value, kc, vc, slots, table, lens, D ** -0.5, Hkv, new_rows_start=starts,
                          partition_size=-1)
        assert torch.equal(got, want)
