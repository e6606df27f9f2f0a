"""Cases of the 4-bit cache and of eviction: what is measured, and each operator's plain form.

Five operators of a serving step over a paged KV cache:

  write       new rows quantised into a 4-bit cache at their slots, then read back as values
  read        rows of a 4-bit or E4M3 cache back as 16-bit values
  decode      single-token attention over a 4-bit cache
  accumulate  single-token attention that also adds every cached token's attention weight
              (summed over the query heads of its KV head) to an fp32 array
  evict       per (sequence, KV head), the most recent tokens and the ones of largest
              accumulated weight move to the front of the sequence's blocks

With ``own`` false, ``run`` computes them with elementary torch operations; with ``own`` true it
makes the calls of the library's binding.

The 4-bit cache: one page per (block of 16 tokens, KV head) of 9 D bytes -- 16 x D/2 bytes of
E2M1 codes, then 16 x D/16 E4M3 scales, one per 16 elements of a token.  With y = x / scale:
sg = E4M3(max(max16 |y| / 6, 2^-9)), code = E2M1(y / sg), value = code sg scale.
"""
import math

import torch

own = False

BLOCK = 16
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's new rows, one per sequence of a batch of 64
        {"name": "write-64-d64", "op": "write", "T": 64, "Hkv": 8, "D": 64, "dtype": "bf16", "pad": 0.0,
         "heads": False},
        # a chunked-prefill step with padding rows, one scale per KV head
        {"name": "write-8192-d128", "op": "write", "T": 8192, "Hkv": 8, "D": 128, "dtype": "bf16", "pad": 0.05,
         "heads": True},
        # a short shared prefix read back from a 4-bit cache for a new prompt's attention
        {"name": "read-333-d128", "op": "read", "T": 333, "Hkv": 4, "D": 128, "dtype": "f16", "cache": "fp4",
         "pad": 0.0, "heads": False},
        # a long history read back whole
        {"name": "read-32768-d128", "op": "read", "T": 32768, "Hkv": 8, "D": 128, "dtype": "bf16", "cache": "fp4",
         "pad": 0.05, "heads": True},
        # two short conversations: latency
        {"name": "decode-2x37-d64", "op": "decode", "S": 2, "Hkv": 4, "G": 1, "D": 64, "Lmin": 5, "Lmax": 37,
         "dtype": "f16", "cache": "fp4"},
        # a batch of 64 conversations, one of them empty (a padded batch) and one of a single token
        {"name": "decode-64x2048-d64", "op": "decode", "S": 64, "Hkv": 8, "G": 4, "D": 64, "Lmin": 0, "Lmax": 2048,
         "dtype": "bf16", "cache": "fp4"},
        # a few very long contexts
        {"name": "decode-4x131072-d128", "op": "decode", "S": 4, "Hkv": 8, "G": 4, "D": 128, "Lmin": 32768,
         "Lmax": 131072, "dtype": "bf16", "cache": "fp4"},
        # a large batch of long contexts
        {"name": "decode-128x8192-d128", "op": "decode", "S": 128, "Hkv": 8, "G": 8, "D": 128, "Lmin": 1024,
         "Lmax": 8192, "dtype": "bf16", "cache": "fp4"},
        # statistics gathered while a batch of 64 decodes over a bf16 cache
        {"name": "accumulate-64x2048-d64", "op": "accumulate", "S": 64, "Hkv": 8, "G": 4, "D": 64, "Lmin": 0,
         "Lmax": 2048, "dtype": "bf16", "cache": "bf16"},
        # the same over a 4-bit cache and longer contexts
        {"name": "accumulate-64x8192-d128", "op": "accumulate", "S": 64, "Hkv": 8, "G": 4, "D": 128, "Lmin": 1024,
         "Lmax": 8192, "dtype": "bf16", "cache": "fp4"},
        # a few conversations that outgrew their budget by a little
        {"name": "evict-5x700-d64", "op": "evict", "S": 5, "Hkv": 4, "D": 64, "Lmin": 400, "Lmax": 700,
         "budget": 512, "recent": 64, "dtype": "f16"},
        # prompts of a batch cut down to a quarter after their prefill
        {"name": "evict-64x4096-d128", "op": "evict", "S": 64, "Hkv": 8, "D": 128, "Lmin": 2048, "Lmax": 4096,
         "budget": 1024, "recent": 128, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "accumulate", "evict"])
    D = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op in ("write", "read"):
        Hkv = rng.choice([1, 2, 4, 5, 8, 16])
        case = {"op": op, "T": _log(rng, 1, 32768 * 8 * 128 // (Hkv * D) // (1 if op == "read" else 4)), "Hkv": Hkv,
                "D": D, "dtype": rng.choice(["bf16", "f16", "f32"]) if op == "write" else dtype,
                "pad": rng.choice([0.0, 0.05, 0.3]), "heads": rng.random() < 0.5}
        if op == "read":
            case["cache"] = rng.choice(["fp4", "fp4", "e4m3"]) if D >= 128 else "fp4"
        return case
    S = _log(rng, 1, 128)
    Hkv = rng.choice([1, 2, 4, 8])
    # elements of one cache at full length, at most the largest listed case's
    most = {"decode": 128 * 8192 * 8 * 128, "accumulate": 64 * 8192 * 8 * 128, "evict": 64 * 4096 * 8 * 128}[op]
    cap = max(16, min({"decode": 131072, "accumulate": 65536, "evict": 32768}[op], most // (S * Hkv * D)))
    Lmax = _log(rng, 16, cap)
    Lmin = rng.choice([0, 1, Lmax // 4, Lmax // 2, Lmax])
    case = {"op": op, "S": S, "Hkv": Hkv, "D": D, "Lmin": Lmin, "Lmax": Lmax, "dtype": dtype}
    if op == "evict":
        budget = max(1, int(Lmax * rng.uniform(0.1, 1.1)))
        case["budget"], case["recent"] = budget, rng.choice([0, 1, budget // 8, budget // 2, budget])
        return case
    case["G"] = rng.choice([1, 2, 3, 4, 6, 8])
    case["cache"] = "fp4" if op == "decode" else rng.choice(["fp4", dtype, "e4m3" if D >= 128 else dtype])
    return case


def _lens(case):
    """Lengths spread evenly over [Lmin, Lmax], in a fixed shuffled order (the same for every seed)."""
    S, lo, hi = case["S"], case["Lmin"], case["Lmax"]
    at = [hi if S == 1 else lo + (hi - lo) * i // (S - 1) for i in range(S)]
    if lo == 0 and S > 2:
        at[1] = 1
    step = next(k for k in (7, 11, 13, 17, 1) if math.gcd(k, S) == 1)
    return [at[i * step % S] for i in range(S)]


def _blocks(L):
    return (L + BLOCK - 1) // BLOCK


def work(case):
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    item = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    if op in ("write", "read"):
        T = case["T"] - int(case["T"] * case["pad"])
        e = T * Hkv * D * 2
        held = 9 / 16 if case.get("cache", "fp4") == "fp4" else 1
        back = min(item, 2)  # what is read back: 16-bit values
        if op == "write":  # rows read, written in 4 bits, read in 4 bits, written as values
            return {"bytes": e * (item + 2 * held + back) + 16 * case["T"], "flops": 4 * e}
        return {"bytes": e * (held + back) + 8 * case["T"], "flops": 2 * e}
    lens = _lens(case)
    if op == "evict":
        kept = sum(min(L, case["budget"]) for L in lens)
        moved = sum(case["budget"] for L in lens if L > case["budget"])
        return {"bytes": Hkv * (4 * sum(lens) + moved * D * item * 2 * 2 + kept * 8), "flops": Hkv * sum(lens)}
    n = sum(lens)
    held = {"fp4": 9 / 16, "e4m3": 1}.get(case["cache"], 2)
    Hq = Hkv * case["G"]
    byts = 2 * n * Hkv * D * held + 2 * case["S"] * Hq * D * item + 4 * sum(map(_blocks, lens)) + 4 * case["S"]
    if op == "accumulate":
        byts += n * Hkv * 8
    return {"bytes": byts, "flops": 4 * n * Hq * D}


# ------------------------------------------------------------------ the 4-bit format, plain

def _page_index(D, device):
    """int64 [16, D/16]: the place of each token's groups' code bytes in a page, in units of 8 bytes
    (a group of 16 elements)."""
    row = min(64, D // 2)
    t = torch.arange(16, device=device)[:, None]
    b = torch.arange(0, D // 2, 8, device=device)[None, :]
    lin = t * row + b % 64
    return ((b // 64) * 1024 + (lin ^ (((lin >> 7) & 3) << 5))) // 8


def _e4m3_round(x):
    return x.clamp(max=448.0).to(torch.float8_e4m3fn)


def _quantise(x, scale):
    """x [..., D], scale broadcast against it: (codes uint8 [..., D], scales uint8 [..., D/16])."""
    y = x.float() / scale
    g = y.unflatten(-1, (-1, 16))
    six = torch.full((), 6.0, device=x.device)  # (a tensor: a plain number would be a product with 1 / 6)
    sg = _e4m3_round((g.abs().amax(-1) / six).clamp(min=2.0 ** -9))
    q = (g / sg.float()[..., None]).abs()
    code = ((q > 0.25).to(torch.uint8) + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5.0))
    code = code + torch.signbit(g).to(torch.uint8) * 8
    return code.flatten(-2), sg.view(torch.uint8)


def _byte_values(device):
    """fp32 [256, 2]: the two E2M1 values of every code byte."""
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=device)
    byte = torch.arange(256, device=device)
    return torch.stack([one[byte & 15], one[byte >> 4]], -1)


def _values(codes8, sg, D, table):
    """Code bytes [..., D/2] and scales uint8 [..., D/16] -> fp32 values [..., D] (without the tensor's scale)."""
    v = torch.index_select(table, 0, codes8.reshape(-1).int()).view(*codes8.shape[:-1], D // 16, 16)
    return (v * sg.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _split_pages(pages, D):
    """Pages [..., 9 D] -> code bytes [..., 16, D/2] in token order, scales [..., 16, D/16]."""
    words = pages[..., : 8 * D].contiguous().view(torch.int64)
    codes = words[..., _page_index(D, pages.device)].view(torch.uint8)
    return codes, pages[..., 8 * D:].unflatten(-1, (16, D // 16))


def _head_scale(scale, Hkv):
    return scale.view(-1, 1) if scale.numel() > 1 else scale.view(1, 1)


# ------------------------------------------------------------------------------- prepare

def _fp4_cache(gen, NB, Hkv, D, device):
    """A pool of pages holding quantised normal values: every group a pick from 65536 quantised ones."""
    bank = torch.randn(1 << 16, 16, generator=gen, device=device)
    codes, sg = _quantise(bank, torch.ones((), device=device))
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous().view(torch.int64).view(-1)
    pick = torch.randint(0, 1 << 16, (NB, Hkv, 16, D // 16), generator=gen, device=device, dtype=torch.int32).long()
    words = torch.empty(NB, Hkv, D, dtype=torch.int64, device=device)
    words[:, :, _page_index(D, device).reshape(-1)] = packed[pick].flatten(2)
    return torch.cat([words.view(torch.uint8), sg.view(-1)[pick].flatten(2)], -1)


def _cache(gen, kind, NB, Hkv, D, device):
    if kind == "fp4":
        return _fp4_cache(gen, NB, Hkv, D, device)
    x = torch.randn(NB, Hkv, BLOCK, D, generator=gen, device=device)
    if kind == "e4m3":
        return (x * 16).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(DT[kind])


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": dict(case), "byte_values": _byte_values(dev)}
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    held = case.get("cache", "fp4" if op in ("write", "read") else case["dtype"])
    one = {"fp4": 1.0, "e4m3": 1.0 / 16}.get(held)
    n_scales = Hkv if case.get("heads") else 1
    for name in ("k_scale", "v_scale"):
        st[name] = None if one is None else one * (0.5 + torch.rand(n_scales, generator=gen, device=dev))
    if op in ("write", "read"):
        T = case["T"]
        NB = _blocks(T) + 4
        slots = torch.randperm(NB * BLOCK, generator=gen, device=dev)[:T]
        slots[torch.randperm(T, generator=gen, device=dev)[: int(T * case["pad"])]] = -1
        st["slots"] = slots
        out = torch.bfloat16 if case["dtype"] == "f32" else DT[case["dtype"]]
        st["key_out"] = torch.zeros(T, Hkv, D, dtype=out, device=dev)
        st["value_out"] = torch.zeros_like(st["key_out"])
        if op == "write":
            # keys: a few channels many times the others' size
            big = 1 + 7 * (torch.rand(Hkv, D, generator=gen, device=dev) < 0.03)
            st["key"] = (torch.randn(T, Hkv, D, generator=gen, device=dev) * big).to(DT[case["dtype"]])
            st["value"] = (torch.randn(T, Hkv, D, generator=gen, device=dev) * 0.3).to(DT[case["dtype"]])
            st["k_cache"] = torch.zeros(NB, Hkv, 9 * D, dtype=torch.uint8, device=dev)
            st["v_cache"] = torch.zeros_like(st["k_cache"])
        else:
            st["k_cache"] = _cache(gen, held, NB, Hkv, D, dev)
            st["v_cache"] = _cache(gen, held, NB, Hkv, D, dev)
        return st
    lens = _lens(case)
    need = [_blocks(L) for L in lens]
    NB, width = sum(need) + max(1, sum(need) // 4), max(need + [1])
    order = torch.randperm(NB, generator=gen, device=dev).int()
    at = torch.tensor([0] + need, device=dev).cumsum(0)
    col = torch.arange(width, device=dev)[None, :]
    held_here = col < torch.tensor(need, device=dev)[:, None]
    st["block_table"] = torch.where(held_here, order[(at[:-1, None] + col).clamp(max=NB - 1)], -1).int()
    st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["k_cache"] = _cache(gen, held, NB, Hkv, D, dev)
    st["v_cache"] = _cache(gen, held, NB, Hkv, D, dev)
    S, W = case["S"], width * BLOCK
    if op != "decode":
        # what earlier steps left: heavy-tailed weights, some tokens never attended to, none at the newest token
        w = torch.exp(1.5 * torch.randn(S, Hkv, W, generator=gen, device=dev))
        w = w * (torch.rand(S, Hkv, W, generator=gen, device=dev) > 0.02)
        last = st["seq_lens"].view(-1, 1, 1) - (0 if op == "evict" else 1)
        st["weights"] = torch.where(torch.arange(W, device=dev) < last, w, 0.0)
    if op == "evict":
        st["kept"] = torch.zeros(S, Hkv, case["budget"], dtype=torch.int32, device=dev)
        st["new_seq_lens"] = torch.zeros(S, dtype=torch.int32, device=dev)
        st["new_weights"] = torch.zeros(S, Hkv, W, device=dev)
        return st
    st["q"] = torch.randn(S, Hkv * case["G"], D, generator=gen, device=dev).to(DT[case["dtype"]])
    st["out"] = torch.zeros_like(st["q"])
    return st


# --------------------------------------------------------------------------- plain forms

def _gathered(cache, st, scale, D):
    """Values of every sequence's tokens, fp32 [S, Hkv, tokens, D] (whatever the padding entries name)."""
    pages = cache[st["block_table"].clamp(min=0)]  # [S, blocks, Hkv, ...]
    if cache.dim() == 3:
        v = _values(*_split_pages(pages, D), D, st["byte_values"])
    elif cache.dtype == torch.uint8:
        v = pages.view(torch.float8_e4m3fn).float()
    else:
        v = pages.float()
    v = v.transpose(1, 2).flatten(2, 3)
    return v if scale is None else v * _head_scale(scale, v.shape[1])[..., None]


def _plain_attention(st):
    case = st["case"]
    S, Hkv, G, D = case["S"], case["Hkv"], case["G"], case["D"]
    k = _gathered(st["k_cache"], st, st["k_scale"], D)
    s = torch.matmul(st["q"].float().view(S, Hkv, G, D) * (1.0 / math.sqrt(D)), k.transpose(2, 3))
    del k
    hidden = (torch.arange(s.shape[-1], device=s.device) >= st["seq_lens"][:, None]).view(S, 1, 1, -1)
    s = s.masked_fill(hidden, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    v = _gathered(st["v_cache"], st, st["v_scale"], D)
    v = v.masked_fill_(hidden.view(S, 1, -1, 1), 0.0)
    st["out"].copy_(torch.matmul(p, v).view(S, Hkv * G, D))
    return p.sum(2)


def _plain_read(st):
    D = st["case"]["D"]
    ok = st["slots"] >= 0
    at = st["slots"].clamp(min=0)
    for cache, scale, out in ((st["k_cache"], st["k_scale"], st["key_out"]),
                              (st["v_cache"], st["v_scale"], st["value_out"])):
        if cache.dim() == 3:
            codes, sg = _split_pages(cache, D)
            rows = _values(codes[at // BLOCK, :, at % BLOCK], sg[at // BLOCK, :, at % BLOCK], D,
                           st["byte_values"])
        else:
            rows = cache[at // BLOCK, :, at % BLOCK].view(torch.float8_e4m3fn).float()
        rows = rows * _head_scale(scale, rows.shape[1])
        out.copy_(torch.where(ok.view(-1, 1, 1), rows.to(out.dtype), out))


def _plain_write(st):
    D = st["case"]["D"]
    ok = st["slots"] >= 0
    at = st["slots"][ok]
    for rows, scale, cache in ((st["key"], st["k_scale"], st["k_cache"]), (st["value"], st["v_scale"], st["v_cache"])):
        codes, sg = _quantise(rows[ok], _head_scale(scale, rows.shape[1]))
        packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).contiguous().view(torch.int64)  # [n, Hkv, D/16]
        words = cache[..., : 8 * D].contiguous().view(torch.int64)
        head = torch.arange(cache.shape[1], device=cache.device).view(1, -1, 1)
        words[(at // BLOCK).view(-1, 1, 1), head, _page_index(D, cache.device)[at % BLOCK][:, None, :]] = packed
        cache[..., : 8 * D] = words.view(torch.uint8)
        cache[..., 8 * D:].unflatten(-1, (16, D // 16))[at // BLOCK, :, at % BLOCK] = sg


def _plain_evict(st):
    case = st["case"]
    S, Hkv, W = st["weights"].shape
    B = case["budget"]
    lens = st["seq_lens"].view(S, 1, 1)
    t = torch.arange(W, device=lens.device)
    recent = (t >= lens - min(case["recent"], B)) & (t < lens)
    key = torch.where(recent, math.inf, torch.where(t < lens, st["weights"], -math.inf))
    best = torch.sort(key, dim=-1, descending=True, stable=True)[1]
    take = min(B, W)
    n = torch.minimum(lens, torch.full_like(lens, B))
    i = torch.arange(take, device=lens.device)
    pos = torch.sort(torch.where(i < n, best[..., :take], W), dim=-1)[0]  # kept positions, ascending; W behind the last
    live = pos < W
    st["kept"].fill_(-1)[..., :take] = torch.where(live, pos, -1).int()
    st["new_seq_lens"].copy_(n.view(-1))
    at = pos.clamp(max=W - 1)
    st["new_weights"].zero_()[..., :take] = torch.where(live, st["weights"].gather(-1, at), 0.0)
    # every row is read before any is written
    s_of, h_of, i_of = live.nonzero(as_tuple=True)
    src, table = at[s_of, h_of, i_of], st["block_table"].long()
    for cache in (st["k_cache"], st["v_cache"]):
        rows = cache[table[s_of, src // BLOCK], h_of, src % BLOCK]
        cache[table[s_of, i_of // BLOCK], h_of, i_of % BLOCK] = rows


def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st)
    if op == "write":
        _plain_write(st)
        _plain_read(st)
        return st["key_out"], st["value_out"]
    if op == "read":
        _plain_read(st)
        return st["key_out"], st["value_out"]
    if op == "decode":
        _plain_attention(st)
        return st["out"]
    if op == "accumulate":
        st["weights"] += _plain_attention(st)
        return st["out"], st["weights"]
    _plain_evict(st)
    return st["kept"], st["new_seq_lens"], st["new_weights"], st["k_cache"], st["v_cache"]


def _run_own(st):
    import paged_decode_attention_reshape_gb300 as pa
    case = st["case"]
    op, Hkv = case["op"], case["Hkv"]
    stride = 1 if case.get("heads") else 0
    if op in ("write", "read"):
        if op == "write":
            pa.pa_reshape_and_cache_opt(st["key"], st["value"], st["k_cache"], st["v_cache"], st["slots"],
                                        pa.PA_KV_FP4_E2M1, k_scale=st["k_scale"], v_scale=st["v_scale"],
                                        scale_stride=stride)
        pa.pa_gather_cache(st["key_out"], st["value_out"], st["k_cache"], st["v_cache"], st["slots"],
                           k_scale=st["k_scale"], v_scale=st["v_scale"], scale_stride=stride)
        return st["key_out"], st["value_out"]
    if op == "evict":
        pa.pa_evict(st["k_cache"], st["v_cache"], st["block_table"], st["seq_lens"], st["weights"], case["budget"],
                    case["recent"], st["kept"], st["new_seq_lens"], st["new_weights"])
        return st["kept"], st["new_seq_lens"], st["new_weights"], st["k_cache"], st["v_cache"]
    scale = 1.0 / math.sqrt(case["D"])
    if op == "decode":
        pa.pa_decode_opt(st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["seq_lens"], scale,
                         Hkv, k_scale=st["k_scale"], v_scale=st["v_scale"])
        return st["out"]
    pa.pa_decode_accumulate(st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["seq_lens"],
                            scale, Hkv, st["weights"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return st["out"], st["weights"]


# ------------------------------------------------------------------- the definition, 64 bits

def _row64(cache, blocks, offs, scale, D):
    """Rows of tokens (block, offset) of every head from their bytes: fp64 [n, Hkv, D]."""
    if cache.dim() == 4:
        c = cache[blocks, :, offs]
        v = (c.view(torch.float8_e4m3fn) if c.dtype == torch.uint8 else c).double()
    else:
        j = torch.arange(D, device=cache.device)
        width = min(64, D // 2)
        lin = offs[:, None] * width + (j // 2)[None, :] % 64
        place = (j // 128)[None, :] * 1024 + (lin ^ (((lin // 128) % 4) * 32))
        n, H = blocks.numel(), cache.shape[1]
        rows = cache[blocks].gather(2, place[:, None, :].expand(n, H, D))
        code = torch.where(j % 2 == 0, rows & 15, rows >> 4).long()
        mag, neg = code % 8, code >= 8
        e, f = mag // 2, mag % 2
        v = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * torch.exp2((e - 1).double()))
        v = torch.where(neg, -v, v)
        where = 8 * D + offs[:, None] * (D // 16) + (j // 16)[None, :]
        sc = cache[blocks].gather(2, where[:, None, :].expand(n, H, D))
        v = v * sc.view(torch.float8_e4m3fn).double()
    if scale is None:
        return v
    return v * (scale.double().view(1, -1, 1) if scale.numel() > 1 else scale.double())


def _exact_quantised(x, scale):
    """The values that rows x [n, Hkv, D] are held as, fp64."""
    sc = scale.double().view(1, -1, 1) if scale.numel() > 1 else scale.double()
    y = (x.double() / sc).float().double()  # a quotient rounded to 64 and then 32 bits is the one rounded to 32
    g = y.view(*y.shape[:-1], -1, 16)
    top = (g.abs().max(-1)[0] / 6).float().clamp(2.0 ** -9, 448.0)
    sg = top.to(torch.float8_e4m3fn).double()[..., None]
    r = (g / sg).float().double()
    mag = r.abs().clamp(max=6.0)
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0)).double()
    mag = torch.round(mag / step) * step  # ties to even multiples of the step
    return (torch.where(r < 0, -mag, mag) * sg).view_as(y) * sc


def exact(case, seed):
    st = prepare(case, seed)
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    if op in ("write", "read"):
        ok = st["slots"] >= 0
        got = []
        for which in ("k", "v"):
            scale = st[which + "_scale"]
            out = torch.zeros(case["T"], Hkv, D, dtype=torch.float64, device=ok.device)
            if op == "write":
                out[ok] = _exact_quantised(st["key" if which == "k" else "value"][ok], scale)
            else:
                at = st["slots"][ok]
                out[ok] = _row64(st[which + "_cache"], at // BLOCK, at % BLOCK, scale, D)
            got.append(out)
        return tuple(got)
    if op == "evict":
        return None  # whole numbers and rows moved bit for bit
    G, S = case["G"], case["S"]
    out = torch.zeros(S, Hkv * G, D, dtype=torch.float64, device="cuda")
    weights = st["weights"].double() if op == "accumulate" else None
    for s, L in enumerate(_lens(case)):
        if L == 0:
            continue
        pos = torch.arange(L, device="cuda")
        blocks, offs = st["block_table"][s, pos // BLOCK].long(), pos % BLOCK
        for h in range(Hkv):
            one = lambda name: _row64(  # noqa: E731
                st[name + "_cache"][:, h:h + 1], blocks, offs, st[name + "_scale"], D)[:, 0]
            q = st["q"][s, h * G:(h + 1) * G].double()
            p = torch.softmax(q @ one("k").T / math.sqrt(D), -1)
            out[s, h * G:(h + 1) * G] = p @ one("v")
            if weights is not None:
                weights[s, h, :L] += p.sum(0)
    return out if weights is None else (out, weights)
