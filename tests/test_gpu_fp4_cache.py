"""The 4-bit cache on the GPU: the write against the fp64 oracle bit for bit, rows read back as
values, block copies.

Tolerances of the read back: a value code * sg * scale is one fp32 product (half a step of fp32,
2^-24 relative) rounded once to the output type (half a step: bf16 2^-8, f16 2^-11 relative; below
f16's smallest normal, half of 2^-24 absolute), so 2^-24 + half a step relative, plus 2^-25."""
import numpy as np
import pytest
import torch

import oracle

import paged_decode_attention_reshape_gb300 as pa

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    pa.lib()
    torch.cuda.set_device(0)


def _rows(T, H, D, dt, seed, edge):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * torch.exp(2 * torch.randn(T, H, 1, generator=g))
    if edge:
        flat = x.view(-1, 16)
        n = flat.shape[0]
        # (groups in range(n) only: small shapes take what fits)
        special = [torch.zeros(16), -torch.zeros(16), torch.full((16,), 1e-30), torch.full((16,), 2.0 ** -9),
                   torch.arange(16) * 0.25 - 2, torch.arange(16) * 0.375, torch.full((16,), 448.0 * 6),
                   torch.full((16,), 3e38), torch.arange(16) * 1e-3, torch.full((16,), 0.25)]
        for i, v in enumerate(special):
            if 3 * i < n:
                flat[3 * i] = v
        for i, bad in enumerate((float("nan"), float("inf"), -float("inf"))):
            if 3 * i + 1 < n:
                flat[3 * i + 1, 5 + i] = bad
        x = flat.view(T, H, D)
    return x.to(dt)


def _write(key, value, kc, vc, slots, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_reshape_and_cache_opt(key, value, kc, vc, slots, pa.PA_KV_FP4_E2M1, device_error=err, **kw)
    return pa.pa_check_device_error(err)


def _expect(pages, slots, x, scale):
    code, sg = oracle.fp4_quantize(x.float().numpy(), scale)
    oracle.fp4_store(pages, slots, code, sg)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 1), (37, 5), (70, 8), (9, 40)])
def test_write_bit_exact(T, H, D, dt):
    NB = (T + 15) // 16 + 3
    key, value = _rows(T, H, D, dt, T + D, True), _rows(T, H, D, dt, T + D + 1, False)
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(NB * 16, generator=g)[:T]
    if T > 5:
        slots[[2, 5]] = -1
    for scale in (None, 0.37, -1.5):
        ref_k = np.full((NB, H, 9 * D), 0xEE, dtype=np.uint8)
        ref_v = ref_k.copy()
        kc, vc = torch.from_numpy(ref_k).cuda(), torch.from_numpy(ref_v).cuda()
        sc = None if scale is None else torch.tensor([scale], device="cuda")
        assert _write(key.cuda(), value.cuda(), kc, vc, slots.cuda(), k_scale=sc, v_scale=sc) == (0, 0)
        s = 1.0 if scale is None else scale
        _expect(ref_k, slots.numpy(), key, s)
        _expect(ref_v, slots.numpy(), value, s)
        assert np.array_equal(kc.cpu().numpy(), ref_k), scale
        assert np.array_equal(vc.cpu().numpy(), ref_v), scale


@pytest.mark.parametrize("scale", [0.0, float("nan"), float("inf"), 2.0 ** -60, 2.0 ** 50])
def test_write_odd_scales(scale):
    T, H, D, NB = 8, 2, 64, 2
    x = _rows(T, H, D, torch.float32, 5, True)
    ref = np.full((NB, H, 9 * D), 0xEE, dtype=np.uint8)
    kc = torch.from_numpy(ref).cuda()
    sc = torch.tensor([scale], device="cuda")
    slots = torch.arange(T)
    assert _write(x.cuda(), x.cuda(), kc, kc.clone(), slots.cuda(), k_scale=sc, v_scale=sc) == (0, 0)
    _expect(ref, slots.numpy(), x, scale)
    assert np.array_equal(kc.cpu().numpy(), ref)


def test_write_ties_of_the_second_quotient():
    """Quotients at and next to every rounding border of E2M1 and E4M3, over many group scales."""
    H, D = 1, 128
    rows = []
    for e in range(0x08, 0x7F):     # every normal E4M3 scale
        s = float(oracle.e4m3_decode([e])[0])
        mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32) * np.float32(s)
        near = np.concatenate([mids, np.nextafter(mids, np.float32(np.inf))])
        rows.append(np.concatenate([near, [6 * s, 0]]))
        rows.append(np.concatenate([np.nextafter(mids, np.float32(0)), mids, [6 * s, -6 * s]]))
    x = np.array(rows, dtype=np.float32)
    x = np.concatenate([x, np.zeros((-len(x) % 8, 16), np.float32)]).reshape(-1, H, D)
    T = x.shape[0]
    NB = (T + 15) // 16
    ref = np.zeros((NB, H, 9 * D), dtype=np.uint8)
    kc = torch.from_numpy(ref).cuda()
    xg = torch.from_numpy(x)
    assert _write(xg.cuda(), xg.cuda(), kc, kc.clone(), torch.arange(T).cuda()) == (0, 0)
    _expect(ref, np.arange(T), xg, 1.0)
    assert np.array_equal(kc.cpu().numpy(), ref)


def test_write_views_and_per_head_scales():
    """Source rows inside a fused [T, 3, H, D] projection, K and V pages interleaved in one
    tensor, scales per head at a stride."""
    T, H, D, NB = 21, 4, 128, 4
    qkv = _rows(T * 3, H, D, torch.bfloat16, 9, False).view(T, 3, H, D).cuda()
    pool = torch.full((NB, 2, H, 9 * D), 0xEE, dtype=torch.uint8, device="cuda")
    heads = np.array([0.05, 0.5, 1.0, 3.0], dtype=np.float32)
    sc = torch.tensor(np.stack([heads, np.full(4, np.nan, np.float32)], 1).ravel(), device="cuda")
    slots = torch.arange(T) * 2 + 3
    assert _write(qkv[:, 1], qkv[:, 2], pool[:, 0], pool[:, 1], slots.cuda(), k_scale=sc, v_scale=sc,
                  scale_stride=2) == (0, 0)
    for i in (0, 1):
        ref = np.full((NB, H, 9 * D), 0xEE, dtype=np.uint8)
        _expect(ref, slots.numpy(), qkv[:, 1 + i].cpu(), heads)
        assert np.array_equal(pool[:, i].cpu().numpy(), ref)


def test_out_of_range_slots():
    T, H, D, NB = 4, 2, 64, 2
    x = _rows(T, H, D, torch.bfloat16, 1, False).cuda()
    kc = torch.full((NB, H, 9 * D), 0xEE, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([0, NB * 16, 2 ** 40, -7], device="cuda")
    vc = kc.clone()
    assert _write(x, x, kc, vc, slots) == (-6, pa.PA_DEVERR_SLOT_RANGE)
    ref = np.full((NB, H, 9 * D), 0xEE, dtype=np.uint8)
    _expect(ref, [0, -1, -1, -1], x.cpu(), 1.0)
    assert np.array_equal(kc.cpu().numpy(), ref)
    out = torch.full_like(x, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_gather_cache(out, out.clone(), kc, vc, slots, device_error=err)
    assert pa.pa_check_device_error(err) == (-6, pa.PA_DEVERR_SLOT_RANGE)
    assert bool((out[1:] == 7.0).all()) and not bool((out[0] == 7.0).all())


@pytest.mark.parametrize("kind", ["fp4", "e4m3", "same"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,D", [(1, 1, 64), (45, 5, 128), (19, 40, 256), (33, 3, 64)])
def test_read_back(T, H, D, dt, kind):
    NB = (T + 15) // 16 + 2
    g = torch.Generator().manual_seed(T * D)
    heads = np.linspace(0.04, 1.7, H).astype(np.float32)
    slots = torch.randint(0, NB * 16, (T,), generator=g)
    if T > 3:
        slots[1], slots[3] = -1, slots[2]      # a hole, and one slot twice
    x = _rows(NB * 16, H, D, torch.float32 if kind != "same" else dt, D, False)
    all_slots = np.arange(NB * 16)
    if kind == "fp4":
        code, sg = oracle.fp4_quantize(x.numpy(), heads)
        pages = np.zeros((NB, H, 9 * D), dtype=np.uint8)
        oracle.fp4_store(pages, all_slots, code, sg)
        cache, vals = torch.from_numpy(pages).cuda(), oracle.fp4_values(code, sg, heads)
    elif kind == "e4m3":
        codes = np.zeros((NB * 16, H, D), dtype=np.uint8)
        oracle.write_flat(x.numpy(), "f32", all_slots, codes, "e4m3", heads)
        cache = torch.from_numpy(codes).view(NB, 16, H, D).transpose(1, 2).contiguous().cuda()
        vals = oracle.cache_values(codes, "e4m3", heads)
    else:
        cache = x.view(NB, 16, H, D).cuda().transpose(1, 2)      # token-major storage
        vals = x.double().numpy()
    sc = torch.tensor(heads, device="cuda")
    key = torch.full((T, H, D), -3.0, dtype=dt, device="cuda")
    wide = torch.full((T, 2, H, D), -3.0, dtype=dt, device="cuda")
    value = wide[:, 1]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_gather_cache(key, value, cache, cache, slots.cuda(), k_scale=sc, v_scale=sc, scale_stride=1,
                       device_error=err)
    assert pa.pa_check_device_error(err) == (0, 0)
    want = vals[slots.clamp(min=0).numpy()]
    for got in (key, value):
        got = got.double().cpu().numpy()
        for t in range(T):
            if slots[t] < 0:
                assert (got[t] == -3.0).all()
            elif kind == "same":
                assert np.array_equal(got[t], want[t])
            else:
                tol = np.abs(want[t]) * (HALF_STEP[dt] + 2.0 ** -24) + (2.0 ** -25 if dt == torch.float16 else 0)
                assert (np.abs(got[t] - want[t]) <= tol).all()
    assert bool((wide[:, 0] == -3.0).all())


def test_copy_blocks_of_pages():
    NB, H, D = 6, 3, 64
    g = torch.Generator().manual_seed(2)
    k = torch.randint(0, 256, (NB, H, 9 * D), generator=g, dtype=torch.uint8)
    v = torch.randint(0, 256, (NB, H, 9 * D), generator=g, dtype=torch.uint8)
    kc, vc = k.cuda(), v.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pairs = torch.tensor([[1, 4], [0, 5], [2, NB]], device="cuda")
    pa.pa_copy_blocks(kc, vc, pairs, err)
    assert pa.pa_check_device_error(err) == (-6, pa.PA_DEVERR_BLOCK_RANGE)
    for ref, got in ((k, kc), (v, vc)):
        ref = ref.clone()
        ref[4], ref[5] = ref[1], ref[0]
        assert torch.equal(ref, got.cpu())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_rows_aligned_to_16_bytes_only(dt):
    """Source and output rows that start 16 bytes off a 32-byte boundary give the same bytes."""
    T, H, D, NB = 50, 3, 64, 5
    x = _rows(T, H, D, dt, 4, True)
    pad = 16 // x.element_size()
    slots = torch.randperm(NB * 16, generator=torch.Generator().manual_seed(1))[:T].cuda()

    def shifted(fill):
        flat = torch.full((T * H * D + pad,), fill, dtype=dt, device="cuda")
        return flat[pad:].view(T, H, D)
    src = shifted(0.0)
    src.copy_(x)
    assert src.data_ptr() % 32 == 16
    pages = []
    for rows in (x.cuda(), src):
        kc = torch.zeros(NB, H, 9 * D, dtype=torch.uint8, device="cuda")
        vc = torch.zeros_like(kc)
        assert _write(rows, rows, kc, vc, slots) == (0, 0)
        assert torch.equal(kc, vc)
        pages.append(kc)
    assert torch.equal(*pages)
    outs = []
    for make in (lambda: torch.zeros(T, H, D, dtype=dt, device="cuda"), lambda: shifted(0.0)):
        key, value = make(), make()
        pa.pa_gather_cache(key, value, pages[0], pages[0], slots)
        outs += [key, value]
    for o in outs[1:]:
        assert torch.equal(outs[0].nan_to_num(7.0), o.nan_to_num(7.0))


def test_read_back_of_many_rows():
    """More rows than one wave of threads."""
    T, H, D, NB = 20011, 8, 128, 40
    g = torch.Generator().manual_seed(11)
    x = _rows(NB * 16, H, D, torch.float32, 3, False)
    code, sg = oracle.fp4_quantize(x.numpy(), 0.7)
    pages = np.zeros((NB, H, 9 * D), dtype=np.uint8)
    oracle.fp4_store(pages, np.arange(NB * 16), code, sg)
    cache = torch.from_numpy(pages).cuda()
    slots = torch.randint(-3, NB * 16, (T,), generator=g)
    want = torch.from_numpy(oracle.fp4_values(code, sg, 0.7)).cuda()[slots.clamp(min=0).cuda()]
    key = torch.full((T, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    value = key.clone()
    pa.pa_gather_cache(key, value, cache, cache, slots.cuda(), k_scale=torch.tensor([0.7], device="cuda"),
                       v_scale=torch.tensor([0.7], device="cuda"))
    gone = (slots < 0).cuda()
    for got in (key, value):
        assert bool((got[gone] == 5.0).all())
        assert bool(((got.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -24))[~gone].all())
