"""pa_rotary and pa_rotary_and_cache on the GPU, against the definitions in 64 bits (rotary_model.py),
and the cache writes bit for bit against pa_rotary followed by pa_reshape_and_cache_opt."""
import pytest
import torch

import paged_decode_attention_reshape_gb300 as pa
import rotary_model as model

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def freqs(R, base=10000.0, **kw):
    return pa.pa_rotary_frequencies(R, base, **kw).to(DEV)


def draw(T, Hq, Hk, D, dtype, seed=0, far=100000, fused=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, Hq + 2 * Hk, D, generator=g).to(dtype).to(DEV)
    pos = torch.randint(0, far, (T,), generator=g).to(DEV)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    return (q, k, v, pos) if fused else (q.contiguous(), k.contiguous(), v.contiguous(), pos)


def weights(D, dtype, seed=5):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.3 * torch.randn(D, generator=g)).to(dtype).to(DEV), (1 + 0.3 * torch.randn(D, generator=g)).to(F32).to(DEV))


SHAPES = [  # T, Hq, Hk
    (1, 1, 1), (1, 32, 8), (7, 5, 1), (37, 3, 3), (130, 8, 2), (65, 64, 8), (300, 1, 1)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 96), (256, 256), (256, 32)])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_rows(dtype, D, R, interleaved):
    for i, (T, Hq, Hk) in enumerate(SHAPES):
        q, k, _, pos = draw(T, Hq, Hk, D, dtype, seed=i)
        f = freqs(R)
        norm = i % 2 == 1
        wq, wk = weights(D, dtype) if norm else (None, None)
        qo, ko = torch.full((T, Hq, D), float("nan"), dtype=dtype, device=DEV), torch.full((T, Hk, D), float("nan"), dtype=dtype, device=DEV)
        m = 1.0 if i % 3 else 1.2079
        pa.pa_rotary(qo, q, ko, k, pos, f, wq, wk, eps=1e-5, interleaved=interleaved, magnitude=m)
        for got, x, w in ((qo, q, wq), (ko, k, wk)):
            want, bound = model.rows(x, pos, f, interleaved, m, w, 1e-5)
            model.assert_rows(got, want, bound, "T %d heads %d/%d" % (T, Hq, Hk))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_and_negative_positions(dtype):
    """Positions through the whole int64 range: the angle is that of the product's part of a turn."""
    pos = torch.tensor([0, 1, -1, 131071, -131072, 1 << 20, (1 << 24) + 1, (1 << 31) + 7, -(1 << 31), 1 << 40, (1 << 62) + 3,
                        -(1 << 63), (1 << 63) - 1], dtype=torch.int64, device=DEV)
    T = len(pos)
    q = torch.randn(T, 2, 128, generator=torch.Generator().manual_seed(3)).to(dtype).to(DEV)
    f = freqs(128)
    out = torch.empty_like(q)
    pa.pa_rotary(out, q, None, None, pos, f)
    model.assert_rows(out, *model.rows(q, pos, f))


def test_int32_positions_are_the_same():
    q, k, _, pos = draw(50, 4, 2, 128, BF, far=1 << 30)
    pos[3] = -5
    a, b = [torch.empty(50, 4, 128, dtype=BF, device=DEV) for _ in range(2)]
    pa.pa_rotary(a, q, None, None, pos, freqs(128))
    pa.pa_rotary(b, q, None, None, pos.int(), freqs(128))
    assert torch.equal(a, b)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_and_side_buffers(dtype, interleaved):
    """In place in the projections' buffer: the same bits, values and everything else untouched."""
    T, Hq, Hk, D, R = 70, 6, 2, 128, 64
    q, k, v, pos = draw(T, Hq, Hk, D, dtype)
    whole = torch.cat((q, k, v), 1)
    padded = torch.cat((whole, whole[:3]), 0).contiguous()
    wq, wk = weights(D, dtype)
    f = freqs(R)
    qo, ko = torch.empty(T, Hq, D, dtype=dtype, device=DEV), torch.empty(T, Hk, D, dtype=dtype, device=DEV)
    pa.pa_rotary(qo, q, ko, k, pos, f, wq, wk, interleaved=interleaved)
    before = padded.clone()
    qi, ki = padded[:T, :Hq], padded[:T, Hq:Hq + Hk]
    pa.pa_rotary(qi, qi, ki, ki, pos, f, wq, wk, interleaved=interleaved)
    assert torch.equal(padded[:T, :Hq], qo) and torch.equal(padded[:T, Hq:Hq + Hk], ko)
    assert torch.equal(padded[:T, Hq + Hk:], before[:T, Hq + Hk:]) and torch.equal(padded[T:], before[T:])


@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_rows_at_16_byte_steps(dtype):
    """Bases and strides that are multiples of 16 bytes and not of 32."""
    T, H, D = 33, 3, 64
    e = 16 // torch.empty(0, dtype=dtype).element_size()
    for interleaved in (False, True):
        g = torch.Generator().manual_seed(1)
        buf = torch.randn(T * (H * (D + e) + 2 * e) + e, generator=g).to(dtype).to(DEV)
        q = torch.as_strided(buf, (T, H, D), (H * (D + e) + 2 * e, D + e, 1), e)
        pos = torch.arange(T, device=DEV) * 997
        out = torch.zeros_like(buf)
        o = torch.as_strided(out, (T, H, D), (H * (D + e) + 2 * e, D + e, 1), e)
        pa.pa_rotary(o, q, None, None, pos, freqs(D), interleaved=interleaved)
        model.assert_rows(o, *model.rows(q, pos, freqs(D), interleaved))
        o.zero_()
        assert not out.any()  # nothing between the rows


def test_broadcast_queries():
    """One query row for all heads and tokens (strides of 0 on an input)."""
    q = torch.randn(128, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV).expand(9, 4, 128)
    pos = torch.arange(9, device=DEV) * 11
    out = torch.empty(9, 4, 128, dtype=BF, device=DEV)
    pa.pa_rotary(out, q, None, None, pos, freqs(128))
    model.assert_rows(out, *model.rows(q, pos, freqs(128)))


def test_norm_without_rotation_and_keys_alone():
    q, k, _, pos = draw(40, 4, 2, 256, F16)
    wq, wk = weights(256, F16)
    out = torch.empty(40, 2, 256, dtype=F16, device=DEV)
    pa.pa_rotary(None, None, out, k, None, None, None, wk)
    model.assert_rows(out, *model.rows(k, None, None, weight=wk))
    copy = torch.empty_like(out)
    pa.pa_rotary(None, None, copy, k, None, None)
    assert torch.equal(copy, k)  # neither norm nor rotation


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_of_extreme_rows(dtype):
    """Rows whose squares pass or vanish below fp32's range are normalised all the same; zeros stay zeros;
    an infinity or a NaN stays in its row."""
    D = 128
    g = torch.Generator().manual_seed(4)
    x = torch.randn(9, 1, D, generator=g)
    for i, by in enumerate((1e30, 1e-30, 3e37, 1e-37, 0.0, 1.0, 1.0, 1e19, 1e-17)):
        x[i] *= by
    x = x.clamp(-3.3e38, 3.3e38)
    x[5, 0, 7] = float("inf")
    x[6, 0, 9] = float("nan")
    q = x.to(dtype).to(DEV)
    w, _ = weights(D, dtype)
    f = freqs(D)
    pos = torch.arange(9, device=DEV)
    out = torch.empty_like(q)
    pa.pa_rotary(out, q, None, None, pos, f, w, eps=0.0)
    want, bound = model.rows(q, pos, f, weight=w, eps=0.0)
    fine = [0, 1, 2, 3, 7, 8]
    model.assert_rows(out[fine], want[fine], bound[fine])
    assert bool(torch.isnan(out[6]).all())
    other = [i for i in range(D) if i not in (7, 7 + D // 2)]
    assert bool((out[5, 0, other] == 0).all()) and bool(torch.isnan(out[5, 0, [7, 7 + D // 2]]).all())
    pa.pa_rotary(out, q, None, None, pos, f, w, eps=1e-6)
    assert not out[4].any()


def test_rotation_composes():
    """Rotating by p and then by -p, or by the way from p to r: two roundings to fp32 from the direct one."""
    q, _, _, p = draw(64, 4, 1, 128, F32)
    r = torch.randint(0, 1 << 20, (64,), generator=torch.Generator().manual_seed(9)).to(DEV)
    f = freqs(128)
    at_p, back, at_r, direct = [torch.empty(64, 4, 128, device=DEV) for _ in range(4)]
    pa.pa_rotary(at_p, q, None, None, p, f)
    pa.pa_rotary(back, at_p, None, None, -p, f)
    pa.pa_rotary(at_r, at_p, None, None, r - p, f)
    pa.pa_rotary(direct, q, None, None, r, f)
    # a rotation is off by 6 u (|a| + |b|) <= 6 sqrt(2) u of the pair's length, and keeps lengths: two 17 u, three 26 u
    pair = lambda x: torch.hypot(x[..., :64], x[..., 64:]).repeat(1, 1, 2)  # noqa: E731
    u = 2.0 ** -24
    assert bool(((back - q).abs() <= 18 * u * pair(q)).all())
    assert bool(((at_r - direct).abs() <= 27 * u * pair(q)).all())


def caches(kind, NB, H, D, dtype, nhd=False):
    if kind == "fp4":
        shape, dt = (NB, H, 9 * D), torch.uint8
    else:
        shape, dt = ((NB, 16, H, D) if nhd else (NB, H, 16, D)), torch.uint8 if kind == "e4m3" else dtype
    c = [torch.full(shape, 0x11, dtype=torch.uint8, device=DEV) if dt is torch.uint8
         else torch.full(shape, 0.125, dtype=dt, device=DEV) for _ in range(2)]
    return [x.permute(0, 2, 1, 3) for x in c] if nhd else c


KV = {"copy": pa.PA_KV_AUTO, "e4m3": pa.PA_KV_FP8_E4M3, "fp4": pa.PA_KV_FP4_E2M1}


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 96), (256, 256), (256, 64), (128, 0)])
@pytest.mark.parametrize("kind", ["copy", "e4m3", "fp4"])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_cache_equals_the_two_calls(dtype, kind, D, R, interleaved):
    for i, (T, Hq, Hk) in enumerate(SHAPES):
        q, k, v, pos = draw(T, Hq, Hk, D, dtype, seed=i, fused=i % 2 == 0)
        f = freqs(R)
        wq, wk = weights(D, dtype) if i % 2 else (None, None)
        NB = T // 16 + 3
        g = torch.Generator().manual_seed(i)
        slots = torch.randperm(NB * 16, generator=g)[:T]
        slots[torch.rand(T, generator=g) < 0.2] = -1
        slots = slots.to(DEV)
        scales, stride = None, 0
        if kind != "copy" and i % 3:
            scales, stride = torch.linspace(0.03, 1.7, Hk, device=DEV), 1 if i % 3 == 1 else 0
        nhd = kind != "fp4" and i % 4 == 2
        opt = dict(k_scale=scales, v_scale=scales, scale_stride=stride)
        rot = dict(eps=1e-6, interleaved=interleaved, magnitude=1.1)
        kc, vc = caches(kind, NB, Hk, D, dtype, nhd)
        qo, ko = torch.empty(T, Hq, D, dtype=dtype, device=DEV), torch.empty(T, Hk, D, dtype=dtype, device=DEV)
        pa.pa_rotary(qo, q, ko, k, pos, f, wq, wk, **rot)
        pa.pa_reshape_and_cache_opt(ko, v, kc, vc, slots, KV[kind], **opt)
        kc2, vc2 = caches(kind, NB, Hk, D, dtype, nhd)
        q2 = torch.full_like(qo, float("nan"))
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        pa.pa_rotary_and_cache(q2, q, k, v, kc2, vc2, pos, slots, f, KV[kind], wq, wk, device_error=err, **rot, **opt)
        assert torch.equal(q2, qo)
        for a, b in ((kc, kc2), (vc, vc2)):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), (T, Hq, Hk)
        assert pa.pa_check_device_error(err) == (0, 0)


@pytest.mark.parametrize("kind", ["copy", "e4m3", "fp4"])
def test_slots_out_of_range(kind):
    """A slot behind the cache writes nothing and sets the error bit; queries are rotated all the same."""
    T, Hq, Hk, D, NB = 20, 4, 2, 128, 2
    q, k, v, pos = draw(T, Hq, Hk, D, BF)
    slots = torch.arange(T, device=DEV) + 1
    slots[4], slots[9] = NB * 16, 1 << 60
    kc, vc = caches(kind, NB, Hk, D, BF)
    kc2, vc2 = caches(kind, NB, Hk, D, BF)
    qo, q2 = torch.empty_like(q), torch.empty_like(q)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_rotary_and_cache(qo, q, k, v, kc, vc, pos, slots, freqs(D), KV[kind], device_error=err)
    assert pa.pa_check_device_error(err) == (-6, pa.PA_DEVERR_SLOT_RANGE)
    ok = slots.clone()
    ok[4] = ok[9] = -1
    pa.pa_rotary_and_cache(q2, q, k, v, kc2, vc2, pos, ok, freqs(D), KV[kind], device_error=err)
    assert pa.pa_check_device_error(err) == (0, 0)
    assert torch.equal(qo, q2) and torch.equal(kc.view(torch.uint8), kc2.view(torch.uint8)) and torch.equal(
        vc.view(torch.uint8), vc2.view(torch.uint8))
    pa.pa_rotary_and_cache(qo, q, k, v, kc, vc, pos, slots, freqs(D), KV[kind])  # no word to set


def test_keys_without_queries_into_the_cache():
    T, Hk, D = 30, 3, 128
    _, k, v, pos = draw(T, 1, Hk, D, BF)
    kc, vc = caches("copy", 3, Hk, D, BF)
    slots = torch.arange(T, device=DEV)
    pa.pa_rotary_and_cache(None, None, k, v, kc, vc, pos, slots, freqs(D))
    rows = kc.permute(0, 2, 1, 3).reshape(-1, Hk, D)
    model.assert_rows(rows[:T], *model.rows(k, pos, freqs(D)))
    assert torch.equal(vc.permute(0, 2, 1, 3).reshape(-1, Hk, D)[:T], v)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (200, 100), (300, 1)])
def test_many_and_few_heads(Hq, Hk):
    """Row counts per token below and above a CTA's range, at a token count that leaves its last range short."""
    T, D = 77, 64
    q, k, v, pos = draw(T, Hq, Hk, D, F16)
    qo, ko = torch.empty(T, Hq, D, dtype=F16, device=DEV), torch.empty(T, Hk, D, dtype=F16, device=DEV)
    pa.pa_rotary(qo, q, ko, k, pos, freqs(D))
    model.assert_rows(qo, *model.rows(q, pos, freqs(D)))
    model.assert_rows(ko, *model.rows(k, pos, freqs(D)))


def test_large_batch_every_row():
    """More rows than one wave of CTAs, a CTA's longest ranges."""
    T, Hq, Hk, D = 3001, 9, 3, 128
    q, k, _, pos = draw(T, Hq, Hk, D, BF, far=4096)
    f = freqs(D)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pa.pa_rotary(qo, q, ko, k, pos, f)
    table = model.angles(torch.arange(4096), f.cpu()).to(DEV)[pos][:, None]
    for got, x in ((qo, q), (ko, k)):
        a, b = x[..., :64].double(), x[..., 64:].double()
        c, s = torch.cos(table), torch.sin(table)
        want = torch.cat((a * c - b * s, b * c + a * s), -1)
        size = (a.abs() + b.abs()).repeat(1, 1, 2)
        bound = 6 * 2.0 ** -24 * size
        bound = bound + 2.0 ** -8 * (want.abs() + bound) + 1e-40
        assert bool(((got.double() - want).abs() <= bound).all())


def test_streams_and_graphs():
    """On a side stream, and captured and replayed over new inputs."""
    T, Hq, Hk, D = 33, 8, 2, 128
    q, k, v, pos = draw(T, Hq, Hk, D, BF, fused=False)
    f = freqs(D)
    wq, wk = weights(D, BF)
    kc, vc = caches("e4m3", 4, Hk, D, BF)
    slots = torch.arange(T, device=DEV)
    qo = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pa.pa_rotary_and_cache(qo, q, k, v, kc, vc, pos, slots, f, KV["e4m3"], wq, wk)
    torch.cuda.current_stream().wait_stream(s)
    want = qo.clone(), kc.clone(), vc.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_rotary_and_cache(qo, q, k, v, kc, vc, pos, slots, f, KV["e4m3"], wq, wk)
    q0, k0, pos0 = q.clone(), k.clone(), pos.clone()
    q.normal_(), k.normal_(), pos.add_(77)
    graph.replay()
    q2, kc2, vc2 = torch.empty_like(q), *caches("e4m3", 4, Hk, D, BF)
    pa.pa_rotary_and_cache(q2, q, k, v, kc2, vc2, pos, slots, f, KV["e4m3"], wq, wk)
    assert torch.equal(qo, q2) and torch.equal(kc, kc2)
    q.copy_(q0), k.copy_(k0), pos.copy_(pos0)
    graph.replay()
    for a, b in zip((qo, kc, vc), want):
        assert torch.equal(a, b)
