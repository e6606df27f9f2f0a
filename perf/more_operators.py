"""Cases of positions and windows: what is measured, and each operator's plain form.

Four operators around a paged KV cache:

  rotary  rows of queries and keys rotated by their positions
  cache   queries and keys normalised per head and rotated, keys and values written into the cache
  decode  single-token attention over the last `window` tokens and the first `sinks` ones
  chunk   the same for several new tokens per sequence

With ``own`` false, ``run`` computes them with elementary torch operations; with ``own`` true it
makes the calls of the library's binding.

Rotation: pair i of a row (elements i and i + R/2, or interleaved 2i and 2i + 1; R the rotated part
of the head) turns by the angle position * theta_i; cos and sin carry the factor `magnitude`.  Norm:
x * rsqrt(mean(x^2) + eps) * weight over the head, before the rotation.  The library's table of
frequencies holds theta_i / (2 pi), turns per position, in units of 2^-64.  A cached key is the rotated
one in the rows' type, converted to the cache's.
"""
import math

import torch

own = False

BLOCK = 16
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch of 64
        {"name": "rotary-64-d64", "op": "rotary", "T": 64, "Hq": 32, "Hkv": 8, "D": 64, "R": 64, "dtype": "bf16",
         "interleaved": False, "far": 2048, "scaled": False},
        # a prompt of odd length, a quarter of wide heads rotated, rows in 32 bits
        {"name": "rotary-777-d256", "op": "rotary", "T": 777, "Hq": 8, "Hkv": 1, "D": 256, "R": 64, "dtype": "f32",
         "interleaved": False, "far": 8192, "scaled": False},
        # a prefill step deep inside long contexts, frequencies scaled for them
        {"name": "rotary-8192-d128", "op": "rotary", "T": 8192, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "dtype": "bf16",
         "interleaved": True, "far": 131072, "scaled": True},
        # one decode step of a batch of 256, heads normalised
        {"name": "cache-256-d128", "op": "cache", "T": 256, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "dtype": "bf16",
         "interleaved": False, "far": 4096, "scaled": False, "norm": True, "cache": "bf16", "pad": 0.0},
        # a step of 64/8 heads into an E4M3 cache, half of the head rotated, padding rows
        {"name": "cache-5001-d128", "op": "cache", "T": 5001, "Hq": 64, "Hkv": 8, "D": 128, "R": 64, "dtype": "bf16",
         "interleaved": True, "far": 8192, "scaled": False, "norm": False, "cache": "e4m3", "pad": 0.05},
        # chunked prefill: 256 sequences x 128 new tokens, heads normalised
        {"name": "cache-32768-d128", "op": "cache", "T": 32768, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "dtype": "bf16",
         "interleaved": False, "far": 4096, "scaled": True, "norm": True, "cache": "bf16", "pad": 0.0},
        # three short conversations, one empty (a padded batch) and one of a single token: latency
        {"name": "decode-3x700-d64", "op": "decode", "S": 3, "Hkv": 4, "G": 1, "D": 64, "Lmin": 0, "Lmax": 700,
         "window": 128, "sinks": 4, "dtype": "f16", "cache": "f16"},
        # a few very long contexts
        {"name": "decode-4x131072-d128", "op": "decode", "S": 4, "Hkv": 8, "G": 4, "D": 128, "Lmin": 32768,
         "Lmax": 131072, "window": 4096, "sinks": 16, "dtype": "bf16", "cache": "bf16"},
        # a large batch, most of it longer than the window
        {"name": "decode-256x4096-d128", "op": "decode", "S": 256, "Hkv": 8, "G": 4, "D": 128, "Lmin": 512,
         "Lmax": 4096, "window": 1024, "sinks": 4, "dtype": "bf16", "cache": "bf16"},
        # 64/8 heads over an E4M3 cache, a window and no sinks
        {"name": "decode-128x8192-d128", "op": "decode", "S": 128, "Hkv": 8, "G": 8, "D": 128, "Lmin": 1024,
         "Lmax": 8192, "window": 2048, "sinks": 0, "dtype": "bf16", "cache": "e4m3"},
        # drafted tokens of five conversations verified at once
        {"name": "chunk-5x7-d64", "op": "chunk", "S": 5, "Hkv": 4, "G": 4, "D": 64, "Lmin": 20, "Lmax": 1000, "nq": 7,
         "window": 256, "sinks": 4, "dtype": "f16", "cache": "f16"},
        # chunked prefill of long prompts
        {"name": "chunk-64x512-d128", "op": "chunk", "S": 64, "Hkv": 8, "G": 4, "D": 128, "Lmin": 512, "Lmax": 8192,
         "nq": 512, "window": 1024, "sinks": 4, "dtype": "bf16", "cache": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "cache", "cache", "decode", "decode", "chunk"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    G = rng.choice([1, 2, 3, 4, 6, 8])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op in ("rotary", "cache"):
        if op == "rotary":
            dtype = rng.choice(["bf16", "f16", "f32"])
        most = (8192 if op == "rotary" else 32768) * 48 * 128 // 2
        case = {"op": op, "T": _log(rng, 1, max(1, most // (Hkv * (G + 2) * D))), "Hq": Hkv * G, "Hkv": Hkv, "D": D,
                "R": rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= D]), "dtype": dtype,
                "interleaved": rng.random() < 0.5, "far": _log(rng, 16, 1 << 20), "scaled": rng.random() < 0.5}
        if op == "cache":
            case["norm"] = rng.random() < 0.6
            case["cache"] = rng.choice([dtype, "e4m3"])
            case["pad"] = rng.choice([0.0, 0.05, 0.3])
        return case
    cache = rng.choice([dtype, dtype, "e4m3"]) if D >= 128 else dtype
    S = _log(rng, 1, 256 if op == "decode" else 64)
    window, sinks = _log(rng, 16, 8192), rng.choice([0, 1, 4, 16, 100])
    nq = 1 if op == "decode" else _log(rng, 2, 512)
    # tokens visible in one sequence: together with the heads no more than the largest listed case's
    cap = {"decode": 256 * 1028 * 8 * 128, "chunk": 64 * 1540 * 8 * 128}[op] // (S * Hkv * D)
    if op == "chunk":
        nq = max(2, min(nq, 64 * 512 * 32 * 128 // (S * Hkv * G * D)))
        cap = min(cap, 64 * 512 * 32 * 1540 * 128 // (S * nq * Hkv * G * D))
    window = max(16, min(window, cap - sinks - nq))
    Lmax = _log(rng, max(16, nq), 131072)
    return {"op": op, "S": S, "Hkv": Hkv, "G": G, "D": D, "Lmin": max(nq if op == "chunk" else 0, rng.choice([0, 1, Lmax // 2, Lmax])),
            "Lmax": Lmax, "window": window, "sinks": sinks, "dtype": dtype, "cache": cache,
            **({"nq": nq} if op == "chunk" else {})}


def _spread(lo, hi, S):
    """S whole numbers spread evenly over [lo, hi], in a fixed shuffled order (the same for every seed)."""
    at = [hi if S == 1 else lo + (hi - lo) * i // (S - 1) for i in range(S)]
    step = next(k for k in (7, 11, 13, 17, 1) if math.gcd(k, S) == 1)
    return [at[i * step % S] for i in range(S)]


def _lens(case):
    S, lo, hi = case["S"], case["Lmin"], case["Lmax"]
    lens = _spread(lo, hi, S)
    if lo == 0 and S > 2:
        lens[lens.index(sorted(lens)[1])] = 1
    return lens


def _news(case):
    """New tokens per sequence: between 1 and nq, never more than the sequence has."""
    return [min(n, L) for n, L in zip(_spread(max(1, case["nq"] // 2), case["nq"], case["S"])[::-1], _lens(case))]


def _seen(L, n, window, sinks):
    """Tokens that the last n queries of a sequence of L see, all together."""
    first = max(0, L - n - window + 1)
    return L if sinks >= first else L - first + sinks


def _pairs(L, n, window, sinks):
    """(query, visible token) pairs of them."""
    return sum(min(p + 1, window) + min(sinks, max(0, p + 1 - window)) for p in range(L - n, L))


def work(case):
    item = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] in ("rotary", "cache"):
        T, Hq, b = case["T"], case["Hq"], item[case["dtype"]]
        rows = T * (Hq + Hkv)
        byts = 2 * T * Hq * D * b + 8 * T
        if case["op"] == "rotary":
            return {"bytes": byts + 2 * T * Hkv * D * b, "flops": rows * 3 * case["R"]}
        kept = T - int(T * case["pad"])
        byts += kept * 2 * Hkv * D * (b + item[case["cache"]]) + 8 * T
        return {"bytes": byts, "flops": rows * (3 * case["R"] + (4 * D if case["norm"] else 0))}
    lens = _lens(case)
    news = [1 if L else 0 for L in lens] if case["op"] == "decode" else _news(case)
    W, K, Hq = case["window"], case["sinks"], Hkv * case["G"]
    seen = sum(_seen(L, n, W, K) for L, n in zip(lens, news) if L)
    rows = sum(news) if case["op"] == "chunk" else case["S"]
    return {"bytes": 2 * seen * Hkv * D * item[case["cache"]] + 2 * rows * Hq * D * item[case["dtype"]] + seen // 4,
            "flops": 4 * D * Hq * sum(_pairs(L, n, W, K) for L, n in zip(lens, news))}


# ------------------------------------------------------------------------------- prepare

def _angles(case):
    """theta_i of the rotated pairs and the magnitude: base 10000, and where scaled, for contexts 8 times
    as long as 4096: pairs that turn less than once over 4096 tokens slowed down by 8, more than 32 times
    left alone, linear in the turns between."""
    R = case["R"]
    theta = [10000.0 ** (-2.0 * i / R) for i in range(R // 2)]
    if not case["scaled"]:
        return theta, 1.0
    keep = [min(1.0, max(0.0, (4096 * t / (2 * math.pi) - 1) / 31)) for t in theta]
    return [t * k + t / 8 * (1 - k) for t, k in zip(theta, keep)], 0.1 * math.log(8.0) + 1.0


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": dict(case)}
    Hkv, D, dt = case["Hkv"], case["D"], DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case["op"] in ("rotary", "cache"):
        T, Hq = case["T"], case["Hq"]
        theta, st["magnitude"] = _angles(case)
        st["theta"] = torch.tensor(theta, dtype=torch.float64, device=dev)
        st["frequencies"] = torch.tensor([round(t / (2 * math.pi) * 2.0 ** 64) for t in theta], dtype=torch.int64, device=dev)
        st["positions"] = torch.randint(0, case["far"], (T,), generator=gen, device=dev)
        # the projections' rows: queries, keys and values side by side
        rows = normal(T, Hq + 2 * Hkv, D).to(dt)
        st["q"], st["key"], st["value"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        st["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device=dev)
        if case["op"] == "rotary":
            st["k_out"] = torch.zeros(T, Hkv, D, dtype=dt, device=dev)
            return st
        NB = (T + BLOCK - 1) // BLOCK + 4
        slots = torch.randperm(NB * BLOCK, generator=gen, device=dev)[:T]
        slots[torch.randperm(T, generator=gen, device=dev)[: int(T * case["pad"])]] = -1
        st["slots"] = slots
        st["q_weight"] = (1 + 0.2 * normal(D)).to(dt) if case["norm"] else None
        st["k_weight"] = (1 + 0.2 * normal(D)).to(dt) if case["norm"] else None
        held = torch.uint8 if case["cache"] == "e4m3" else dt
        st["k_cache"] = torch.zeros(NB, Hkv, BLOCK, D, dtype=held, device=dev)
        st["v_cache"] = torch.zeros_like(st["k_cache"])
        for name in ("k_scale", "v_scale"):
            st[name] = (0.5 + torch.rand(1, generator=gen, device=dev)) / 16 if case["cache"] == "e4m3" else None
        return st

    lens = _lens(case)
    news = [1] * case["S"] if case["op"] == "decode" else _news(case)
    W, K = case["window"], case["sinks"]
    # blocks that no query sees any more have been given back: their entries are -1
    held = []
    for L, n in zip(lens, news):
        first = max(0, L - n - W + 1) // BLOCK
        held.append([b for b in range((L + BLOCK - 1) // BLOCK) if b >= first or b * BLOCK < K])
    NB, width = max(1, sum(map(len, held))), max([(L + BLOCK - 1) // BLOCK for L in lens] + [1])
    order = torch.randperm(NB, generator=gen, device=dev).int()
    at = torch.tensor([s * width + b for s, bs in enumerate(held) for b in bs], dtype=torch.int64, device=dev)
    table = torch.full((case["S"] * width,), -1, dtype=torch.int32, device=dev)
    table[at] = order[: at.numel()]
    st["block_table"] = table.view(case["S"], width)
    st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    for name in ("k", "v"):
        x = normal(NB, Hkv, BLOCK, D)
        st[name + "_cache"] = (x * 16).to(torch.float8_e4m3fn).view(torch.uint8) if case["cache"] == "e4m3" else x.to(dt)
        st[name + "_scale"] = (0.5 + torch.rand(1, generator=gen, device=dev)) / 16 if case["cache"] == "e4m3" else None
    rows = case["S"] if case["op"] == "decode" else sum(news)
    st["q"] = normal(rows, Hkv * case["G"], D).to(dt)
    st["out"] = torch.zeros_like(st["q"])
    if case["op"] == "chunk":
        st["query_start_loc"] = torch.tensor([0] + news, device=dev).cumsum(0).int()
    return st


# --------------------------------------------------------------------------- plain forms

def _plain_rows(st, x, weight):
    """Rows x [T, H, D] normalised (with a weight) and rotated, fp32."""
    case = st["case"]
    R = case["R"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    angle = st["positions"].double()[:, None, None] * st["theta"]
    cos, sin = (torch.cos(angle) * st["magnitude"]).float(), (torch.sin(angle) * st["magnitude"]).float()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if case["interleaved"] else (x[..., : R // 2], x[..., R // 2: R])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., R:]), -1)


def _plain_stored(cache, scale, rows, slots):
    """Rows of the cache's values put at their slots."""
    if scale is not None:
        rows = (rows.float() / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    ok = slots >= 0
    cache[slots[ok] // BLOCK, :, slots[ok] % BLOCK] = rows[ok]


def _plain_attention(st):
    """Queries padded to [S, n], each sequence's visible tokens gathered: the first `sinks`, and those from
    the first query's window on."""
    case = st["case"]
    S, Hkv, G, D, W, K = (case[k] for k in ("S", "Hkv", "G", "D", "window", "sinks"))
    n = case.get("nq", 1)
    dev = st["q"].device
    L = st["seq_lens"].long()
    if case["op"] == "decode":
        start, new = torch.arange(S, device=dev), torch.ones(S, dtype=torch.int64, device=dev)
    else:
        start, new = st["query_start_loc"][:-1].long(), st["query_start_loc"].long().diff()
    i = torch.arange(n, device=dev)
    row = torch.where(i < new[:, None], start[:, None] + i, start[:, None])
    pos = (L - new)[:, None] + i  # [S, n]
    tail = torch.arange(n + W - 1, device=dev) + (L - new - W + 1)[:, None]
    t = torch.cat((torch.arange(K, device=dev).expand(S, K), torch.where(tail >= K, tail, -1)), 1)  # -1: no token
    t = torch.where(t < L[:, None], t, -1)
    sees = (t[:, None] >= 0) & (t[:, None] <= pos[:, :, None]) & ((t[:, None] > pos[:, :, None] - W) | (t[:, None] < K))
    at = t.clamp(min=0)
    block, off = st["block_table"].gather(1, at // BLOCK).clamp(min=0).long(), at % BLOCK

    def values(name):
        rows = st[name + "_cache"][block, :, off]  # [S, tokens, Hkv, D]
        scale = st[name + "_scale"]
        rows = rows.float() if scale is None else rows.view(torch.float8_e4m3fn).float() * scale
        return rows.masked_fill_((t < 0)[..., None, None], 0.0).transpose(1, 2)

    q = st["q"].float()[row].view(S, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * n, D)
    s = torch.matmul(q * (1.0 / math.sqrt(D)), values("k").transpose(2, 3)).view(S, Hkv, G, n, -1)
    s = s.masked_fill(~sees[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    o = torch.matmul(p.view(S, Hkv, G * n, -1), values("v")).view(S, Hkv, G, n, D)
    o = o.permute(0, 3, 1, 2, 4).reshape(S, n, Hkv * G, D).to(st["out"].dtype)
    live = i < new[:, None]
    st["out"][row[live]] = o[live]


def run(st):
    case = st["case"]
    if own:
        return _run_own(st)
    if case["op"] == "rotary":
        st["q_out"].copy_(_plain_rows(st, st["q"], None))
        st["k_out"].copy_(_plain_rows(st, st["key"], None))
        return st["q_out"], st["k_out"]
    if case["op"] == "cache":
        st["q_out"].copy_(_plain_rows(st, st["q"], st["q_weight"]))
        key = _plain_rows(st, st["key"], st["k_weight"]).to(st["key"].dtype)
        _plain_stored(st["k_cache"], st["k_scale"], key, st["slots"])
        _plain_stored(st["v_cache"], st["v_scale"], st["value"], st["slots"])
        return _cached(st)
    _plain_attention(st)
    return st["out"]


def _cached(st):
    held = (st["k_cache"], st["v_cache"])
    if st["case"]["cache"] == "e4m3":
        held = tuple(c.view(torch.float8_e4m3fn) for c in held)
    return st["q_out"], *held


def _run_own(st):
    import paged_decode_attention_reshape_gb300 as pa
    case = st["case"]
    if case["op"] == "rotary":
        pa.pa_rotary(st["q_out"], st["q"], st["k_out"], st["key"], st["positions"], st["frequencies"],
                     interleaved=case["interleaved"], magnitude=st["magnitude"])
        return st["q_out"], st["k_out"]
    if case["op"] == "cache":
        pa.pa_rotary_and_cache(st["q_out"], st["q"], st["key"], st["value"], st["k_cache"], st["v_cache"],
                               st["positions"], st["slots"], st["frequencies"],
                               pa.PA_KV_FP8_E4M3 if case["cache"] == "e4m3" else pa.PA_KV_AUTO,
                               q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                               interleaved=case["interleaved"], magnitude=st["magnitude"],
                               k_scale=st["k_scale"], v_scale=st["v_scale"])
        return _cached(st)
    scale = 1.0 / math.sqrt(case["D"])
    if case["op"] == "decode":
        pa.pa_decode_window(st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["seq_lens"],
                            scale, case["Hkv"], case["window"], case["sinks"], k_scale=st["k_scale"],
                            v_scale=st["v_scale"])
    else:
        pa.pa_attention_window(st["out"], st["q"], st["k_cache"], st["v_cache"], st["query_start_loc"],
                               st["block_table"], st["seq_lens"], scale, case["Hkv"], case["nq"], case["window"],
                               case["sinks"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return st["out"]


# ------------------------------------------------------------------- the definition, 64 bits

def _exact_rows(st, x, weight):
    case = st["case"]
    R, D = case["R"], case["D"]
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * weight.double()
    out = x.clone()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
        angle = st["positions"].double() * st["theta"][i]
        c, s = (torch.cos(angle) * st["magnitude"])[:, None], (torch.sin(angle) * st["magnitude"])[:, None]
        out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        out[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return out


def _exact_stored(st, name, rows):
    """The values that the whole cache holds without rounding, rows [T, Hkv, D] (fp64) at their slots."""
    cache, scale = st[name + "_cache"], st[name + "_scale"]
    if scale is not None:
        rows = (rows / scale.double()).clamp(-448.0, 448.0)
    out = torch.zeros(cache.shape, dtype=torch.float64, device=cache.device)
    ok = (st["slots"] >= 0).nonzero()[:, 0]
    out[st["slots"][ok] // BLOCK, :, st["slots"][ok] % BLOCK] = rows[ok]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rows(st, st["q"], None), _exact_rows(st, st["key"], None)
    if case["op"] == "cache":
        return (_exact_rows(st, st["q"], st["q_weight"]),
                _exact_stored(st, "k", _exact_rows(st, st["key"], st["k_weight"])),
                _exact_stored(st, "v", st["value"].double()))
    lens, S, Hkv, G, D = _lens(case), case["S"], case["Hkv"], case["G"], case["D"]
    news = [1] * S if case["op"] == "decode" else _news(case)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for s, (L, n) in enumerate(zip(lens, news)):
        first = max(0, L - n - case["window"] + 1)
        sinks = min(case["sinks"], first)
        t = torch.cat((torch.arange(sinks, device="cuda"), torch.arange(first, L, device="cuda")))
        if L == 0:
            row += n
            continue
        block, off = st["block_table"][s, t // BLOCK].long(), t % BLOCK
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        hidden = (t > pos) | ((t <= pos - case["window"]) & (t >= case["sinks"]))
        for g in range(Hkv):
            def rows(name):
                x = st[name + "_cache"][:, g][block, off]
                scale = st[name + "_scale"]
                return x.double() if scale is None else x.view(torch.float8_e4m3fn).double() * scale.double()
            k, v = rows("k"), rows("v")
            for h in range(g * G, (g + 1) * G):
                z = st["q"][row:row + n, h].double() @ k.T / math.sqrt(D)
                out[row:row + n, h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v
        row += n
    return out
