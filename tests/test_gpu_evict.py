"""pa_evict on the GPU, every output bit for bit against a plain selection and move in numpy, and the
whole cycle: 4-bit writes, decodes that accumulate weights, eviction, blocks given back, decode."""
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


def keep(w, L, budget, recent):
    """Positions kept of one row: the last tokens, and the largest of the others, ties by position."""
    if L <= budget:
        return np.arange(L)
    r = min(recent, budget)
    cand = L - r
    key = np.where(np.isnan(w[:cand]), -np.inf, w[:cand]).astype(np.float64)
    # NaN below -inf: (is a number, value) descending, position ascending
    order = np.lexsort((np.arange(cand), -key, np.isnan(w[:cand])))
    return np.sort(np.concatenate([order[:budget - r], np.arange(cand, L)]).astype(np.int64))


ROWB = {"bf16": lambda D: 2 * D, "f16": lambda D: 2 * D, "f32": lambda D: 4 * D, "e4m3": lambda D: D}
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.uint8}


class Setup:
    def __init__(self, kind, H, D, lens, seed=0, layout="hnd", extra=3):
        rng = np.random.RandomState(seed)
        self.kind, self.H, self.D, self.lens = kind, H, D, np.array(lens, np.int32)
        need = (self.lens + 15) // 16
        self.NB, self.MB = int(need.sum()) + 4, int(max(need.max(), 1)) + 1
        self.W = self.MB * 16 + extra
        order = rng.permutation(self.NB)
        self.table = np.full((len(lens), self.MB), -7, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        rb = 9 * D // 16 if kind == "fp4" else ROWB[kind](D)
        # rows [K / V, slot, head, bytes] as bytes
        self.rows = rng.randint(0, 256, (2, self.NB * 16, H, rb)).astype(np.uint8)
        if kind == "fp4":
            place = oracle.fp4_place(D)
            pool = np.zeros((2, self.NB, H, 9 * D), np.uint8)
            r = self.rows.reshape(2, self.NB, 16, H, rb)
            for t in range(16):
                pool[..., place[t]] = r[:, :, t]
            self.cache = [torch.from_numpy(pool[i]).cuda() for i in (0, 1)]
        else:
            r = self.rows.reshape(2, self.NB, 16, H, rb)
            if layout == "nhd":
                self.cache = [torch.from_numpy(r[i].copy()).cuda().view(DT[kind]).transpose(1, 2) for i in (0, 1)]
            else:
                self.cache = [torch.from_numpy(r[i].transpose(0, 2, 1, 3).copy()).cuda().view(DT[kind]) for i in (0, 1)]
        self.weights = np.exp(rng.randn(len(lens), H, self.W)).astype(np.float32)

    def slot(self, s, pos):
        return self.table[s][pos // 16].astype(np.int64) * 16 + pos % 16

    def bytes_now(self):
        out = np.zeros_like(self.rows)
        for i, c in enumerate(self.cache):
            if self.kind == "fp4":
                place = oracle.fp4_place(self.D)
                page = c.cpu().numpy()
                r = np.stack([page[..., place[t]] for t in range(16)], 1)       # [NB, 16, H, rb]
            else:
                t = c.transpose(1, 2).contiguous().cpu()                        # [NB, 16, H, D]
                r = t.view(torch.uint8).numpy() if t.dtype != torch.uint8 else t.numpy()
            out[i] = r.reshape(self.NB * 16, self.H, -1)
        return out

    def run(self, budget, recent, seq_lens=None, table=None):
        S = len(self.lens)
        kept = torch.full((S, self.H, budget), 99, dtype=torch.int32, device="cuda")
        nl = torch.full((S,), 99, dtype=torch.int32, device="cuda")
        nw = torch.full((S, 2, self.H, self.W), 9.0, device="cuda")[:, 1]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.pa_evict(self.cache[0], self.cache[1], torch.from_numpy(self.table if table is None else table).cuda(),
                    torch.from_numpy(self.lens if seq_lens is None else seq_lens).cuda(),
                    torch.from_numpy(self.weights).cuda(), budget, recent, kept, nl, nw, device_error=err)
        return pa.pa_check_device_error(err), kept.cpu().numpy(), nl.cpu().numpy(), nw.cpu().numpy()

    def check(self, budget, recent, got, untouched=()):
        (rc, bits), kept, nl, nw = got
        assert (rc, bits) == (0, 0) or untouched
        rows = self.rows.copy()
        for s, L in enumerate(self.lens):
            if s in untouched:
                continue
            for h in range(self.H):
                pos = keep(self.weights[s, h], int(L), budget, recent)
                n = len(pos)
                assert np.array_equal(kept[s, h], np.concatenate([pos, np.full(budget - n, -1)])), (s, h)
                want = np.zeros(self.W, np.float32)
                want[:n] = self.weights[s, h, pos]
                assert np.array_equal(nw[s, h], want, equal_nan=True), (s, h)
                if L > budget:
                    rows[:, self.slot(s, np.arange(n)), h] = self.rows[:, self.slot(s, pos), h]
            assert nl[s] == min(L, budget)
        assert np.array_equal(self.bytes_now(), rows)


CASES = [("bf16", 4, 64), ("f16", 1, 128), ("bf16", 3, 256), ("f32", 2, 64), ("f32", 1, 256), ("e4m3", 4, 128),
         ("fp4", 4, 64), ("fp4", 3, 128), ("fp4", 2, 256), ("bf16", 2, 8), ("bf16", 3, 24)]


@pytest.mark.parametrize("kind,H,D", CASES, ids=["%s-%d-%d" % c for c in CASES])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (16, 0), (100, 7), (129, 129), (200, 1000), (700, 64)])
def test_bit_exact(kind, H, D, budget, recent):
    s = Setup(kind, H, D, [0, 1, 16, 100, 129, 130, 701, 1500], seed=budget + D)
    s.check(budget, recent, s.run(budget, recent))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_token_major_caches(kind):
    s = Setup(kind, 5, 128, [300, 40, 77], seed=1, layout="nhd")
    s.check(50, 10, s.run(50, 10))


def test_special_weights():
    """Ties, zeros of both signs, infinities, NaN, negative and subnormal weights."""
    s = Setup("bf16", 6, 64, [900, 900], seed=2)
    w = s.weights
    w[:, 0] = 0.5                                                    # all equal: the lowest positions
    w[:, 1] = np.where(np.arange(s.W) % 2, 0.0, -0.0)                # -0 equals +0
    w[:, 2, ::3] = np.nan
    w[:, 3, ::5], w[:, 3, 1::5] = np.inf, -np.inf
    w[:, 4] = (np.arange(s.W) % 7).astype(np.float32) * 1e-42
    w[:, 5] = -w[:, 5]
    w[1, 2] = np.nan                                                 # nothing but NaN
    for budget, recent in ((64, 0), (250, 30), (700, 1)):
        t = Setup("bf16", 6, 64, [900, 900], seed=2)
        t.weights = w
        t.check(budget, recent, t.run(budget, recent))


def test_rows_already_in_place_and_far_moves():
    s = Setup("f16", 2, 128, [2000, 2000], seed=3)
    s.weights[:, 0] = -np.arange(s.W)                                # the first tokens: nothing moves
    s.weights[:, 1] = np.arange(s.W)                                 # the last tokens: everything moves by 1000
    s.check(1000, 0, s.run(1000, 0))


def test_long_row():
    s = Setup("fp4", 2, 64, [70000], seed=4)
    s.check(20000, 500, s.run(20000, 500))


def test_many_heads_and_sequences():
    s = Setup("bf16", 40, 64, [33 + 3 * i for i in range(30)], seed=5)
    s.check(64, 8, s.run(64, 8))


def test_faults_leave_the_sequence():
    s = Setup("fp4", 2, 128, [300, 200, 260, 250], seed=6)
    table, lens = s.table.copy(), s.lens.copy()
    table[1, 12] = s.NB                      # the last used entry
    table[3, 0] = -1
    lens[2] = s.MB * 16 + 1
    got = s.run(100, 20, lens, table)
    assert got[0] == (-6, pa.PA_DEVERR_BLOCK_RANGE | pa.PA_DEVERR_SEQLEN_RANGE)
    s.check(100, 20, got, untouched=(1, 2, 3))
    _, kept, nl, nw = got
    for i in (1, 2, 3):
        assert (kept[i] == -1).all() and nl[i] == lens[i] and np.array_equal(nw[i], s.weights[i])


def test_captured():
    s = Setup("bf16", 2, 64, [500, 90], seed=7)
    bt, sl, w = (torch.from_numpy(x).cuda() for x in (s.table, s.lens, s.weights))
    kept = torch.zeros(2, 2, 100, dtype=torch.int32, device="cuda")
    nl, nw = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros_like(w)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pa.pa_evict(s.cache[0], s.cache[1], bt, sl, w, 100, 10, kept, nl, nw)
    torch.cuda.synchronize()
    assert np.array_equal(s.bytes_now(), s.rows)
    graph.replay()
    torch.cuda.synchronize()
    s.check(100, 10, ((0, 0), kept.cpu().numpy(), nl.cpu().numpy(), nw.cpu().numpy()))


@pytest.mark.parametrize("D", [64, 128])
def test_generation_under_a_budget(D):
    """Two sequences grow token by token in a 4-bit cache; every step writes, attends and accumulates;
    whenever a sequence passes 48 tokens it is cut to 32 and its blocks go back to the pool.  Outputs of
    every step are checked against the tokens that the kept positions say are still there."""
    Hq, H, S, budget, recent = 8, 2, 2, 32, 6
    G = Hq // H
    bm = pa.BlockManager(9, S, 4)                       # 9 blocks: not enough for both without eviction
    kc = torch.zeros(9, H, 9 * D, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    weights = torch.zeros(S, H, 64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rng = np.random.RandomState(D)
    vals = [[[[] for _ in range(H)] for _ in range(2)] for _ in range(S)]       # [seq][K / V][head] -> rows
    scale, evictions = D ** -0.5, 0
    for step in range(110):
        rows = rng.randn(2, S, H, D).astype(np.float32)
        x = torch.from_numpy(rows).to(torch.bfloat16)
        slots = np.array([bm.append(s, 1)[0][0] for s in range(S)])
        pa.pa_reshape_and_cache(x[0].cuda(), x[1].cuda(), kc, vc, torch.from_numpy(slots).cuda(), pa.PA_KV_FP4_E2M1,
                                device_error=err)
        for i in (0, 1):
            held = oracle.fp4_values(*oracle.fp4_quantize(x[i].float().numpy(), 1.0))
            for s in range(S):
                for h in range(H):
                    vals[s][i][h].append(held[s, h])
        bt, sl = (torch.from_numpy(a).cuda() for a in bm.export([0, 1]))
        q = torch.from_numpy(rng.randn(S, Hq, D).astype(np.float32)).to(torch.bfloat16)
        out = torch.full((S, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        pa.pa_decode_accumulate(out, q.cuda(), kc, vc, bt, sl, scale, H, weights, device_error=err)
        c = fp4_cases.Fp4Case()
        c.S, c.Hq, c.Hkv, c.D, c.nq, c.alibi, c.q, c.scale, c.dtype = S, Hq, H, D, None, None, q, scale, torch.bfloat16
        c.lens = sl.tolist()
        c.K, c.V = ([np.stack([np.stack(vals[s][i][h]) for h in range(H)], 1) for s in range(S)] for i in (0, 1))
        ref, tol, _ = fp4_cases.reference(c)
        fp4_cases.check(out, ref, tol, "step %d" % step)
        if max(c.lens) > 48:
            kept = torch.zeros(S, H, budget, dtype=torch.int32, device="cuda")
            nl, nw = torch.zeros_like(sl), torch.zeros_like(weights)
            w = weights.cpu().numpy()
            pa.pa_evict(kc, vc, bt, sl, weights, budget, recent, kept, nl, nw, device_error=err)
            for s in range(S):
                for h in range(H):
                    pos = keep(w[s, h], c.lens[s], budget, recent)
                    assert np.array_equal(kept[s, h].cpu().numpy(), pos)
                    for i in (0, 1):
                        vals[s][i][h] = [vals[s][i][h][p] for p in pos]
                bm.truncate(s, int(nl[s]))
            weights = nw
            evictions += 1
        assert pa.pa_check_device_error(err) == (0, 0)
    assert evictions >= 4 and G == 4


def test_empty_tables():
    """A batch whose table has no columns: every length is 0 and every output is written."""
    kc = torch.zeros(2, 3, 16, 64, dtype=torch.bfloat16, device="cuda")
    sl = torch.tensor([0, 0, 5], dtype=torch.int32, device="cuda")
    kept = torch.full((3, 3, 4), 9, dtype=torch.int32, device="cuda")
    nl = torch.full((3,), 9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for W in (0, 7):
        w = torch.ones(3, 3, W, device="cuda")
        nw = torch.full_like(w, 9.0)
        pa.pa_evict(kc, kc.clone(), torch.zeros(3, 0, dtype=torch.int32, device="cuda"), sl, w, 4, 1, kept, nl, nw,
                    device_error=err)
        assert pa.pa_check_device_error(err) == (-6, pa.PA_DEVERR_SEQLEN_RANGE)
        assert bool((kept == -1).all()) and nl.tolist() == [0, 0, 5]
        assert not bool(nw[:2].any()) and bool((nw[2] == 1).all())


@pytest.mark.parametrize("kind,H,D", [("bf16", 1, 128), ("f32", 2, 64), ("e4m3", 1, 128), ("fp4", 2, 128), ("fp4", 1, 64), ("fp4", 1, 256)])
@pytest.mark.parametrize("lens,budget,recent", [([20011, 4100], 6000, 100), ([16385], 1025, 1024), ([9000, 8191, 0, 1], 4097, 0)])
def test_few_long_sequences(kind, H, D, lens, budget, recent):
    """More tokens than a thread's registers hold, few CTAs: the wide forms of both kernels."""
    s = Setup(kind, H, D, lens, seed=11)
    s.weights[:, :, 17:9000:3] = np.float32(0.25)               # many equal weights around the threshold
    s.weights[0, 0, 5:50] = [np.nan, np.inf, -np.inf, 0.0, -0.0] * 9
    s.check(budget, recent, s.run(budget, recent))


def test_few_long_sequences_stay_below_the_wide_forms():
    """As many pairs as SMs and more: 256 threads again, same answer."""
    for H, lens in ((8, [5000] * 3), (8, [5000] * 24)):
        s = Setup("bf16", H, 64, lens, seed=12)
        s.check(1500, 64, s.run(1500, 64))
