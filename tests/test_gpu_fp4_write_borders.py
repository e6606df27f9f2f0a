"""The 4-bit write where quotients meet rounding borders: every significand of a group's largest element,
the other elements on or next to the codes' borders, at head scales that 16-bit rows meet borders with
often (none given, powers of two, few bits) and others.  Bit for bit against the oracle; and no scale
that a caller may have is many times slower than another."""
import numpy as np
import pytest
import torch

import oracle

import paged_decode_attention_reshape_gb300 as pa

pytestmark = pytest.mark.gpu

SCALES = [None, 0.5, 0.0625, -2.0, 0.75, 1.5, 3.0, 0.8371, -0.37, 1.0 / 3, 2.0 ** -20, 2.0 ** 39, 1.75 * 2.0 ** -39]
H, D = 8, 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    pa.lib()
    torch.cuda.set_device(0)


def _tops(dt, rng):
    """Largest elements: all significands at many exponents (fp32: random ones, and the borders' own)."""
    if dt is torch.bfloat16:
        sig, exps = 1 + np.arange(128) / 128, range(-14, 14)
    elif dt is torch.float16:
        sig, exps = 1 + np.arange(1024) / 1024, range(-13, 14, 3)
    else:
        sig, exps = np.concatenate([1 + rng.rand(512), 1 + np.arange(64) / 64]).astype(np.float32), range(-14, 14, 3)
    return np.concatenate([sig * 2.0 ** e for e in exps]).astype(np.float32)


def _groups(dt, scale, rng):
    s = np.float64(1.0 if scale is None else np.float32(scale))
    top = _tops(dt, rng)
    if dt is not torch.float16:       # (in f16's range as they are)
        top = (top * 2.0 ** np.floor(np.log2(abs(s)))).astype(np.float32)
    x = rng.uniform(-1, 1, (len(top), 16)).astype(np.float32) * top[:, None]
    _, sg = oracle.fp4_quantize(np.broadcast_to(top[:, None, None], (len(top), 1, 16)), np.float32(s))
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -2.5, -5.0])
    on = border * oracle.e4m3_decode(sg[:, 0, 0])[:, None] * s
    x[:, 1:12] = np.where(np.abs(on) <= top[:, None], on, x[:, 1:12])
    x[:, 12] = -0.0
    x[:, 0] = top * rng.choice([-1, 1], len(top))
    for i in range(len(x)):
        x[i] = rng.permutation(x[i])
    x = np.concatenate([x, np.zeros((-len(x) % (H * D // 16), 16), np.float32)])
    return torch.from_numpy(x.reshape(-1, H, D)).to(dt)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "f16", "f32"])
def test_bit_exact(dt, scale):
    x = _groups(dt, scale, np.random.RandomState(1))
    T, NB = x.shape[0], (x.shape[0] + 15) // 16
    ref = np.zeros((NB, H, 9 * D), dtype=np.uint8)
    code, sg = oracle.fp4_quantize(x.float().numpy(), 1.0 if scale is None else scale)
    oracle.fp4_store(ref, np.arange(T), code, sg)
    kc = torch.zeros(NB, H, 9 * D, dtype=torch.uint8, device="cuda")
    vc, sc = kc.clone(), None if scale is None else torch.tensor([scale], device="cuda")
    pa.pa_reshape_and_cache_opt(x.cuda(), x.cuda(), kc, vc, torch.arange(T).cuda(), pa.PA_KV_FP4_E2M1, k_scale=sc,
                                v_scale=sc)
    assert np.array_equal(kc.cpu().numpy(), ref) and torch.equal(kc, vc)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_no_scale_is_many_times_slower(dt):
    """Normal rows: the best of a few replays at each scale within 4 times that at 0.8371 (dividing in
    loops out of local memory took 8 to 15 times)."""
    T = 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, D, generator=g, device="cuda").to(dt)
    kc = torch.zeros(T // 16, H, 9 * D, dtype=torch.uint8, device="cuda")
    vc, slots = kc.clone(), torch.arange(T, device="cuda")
    best = {}
    for scale in (0.8371, None, 0.5, 0.75, 0.0625):
        sc = None if scale is None else torch.tensor([scale], device="cuda")
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(10):
                pa.pa_reshape_and_cache_opt(x, x, kc, vc, slots, pa.PA_KV_FP4_E2M1, k_scale=sc, v_scale=sc)
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            graph.replay()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        best[scale] = min(times)
    assert all(t < 4 * best[0.8371] for t in best.values()), best
