"""Rotation, norm and their tolerances in 64 bits, from the definitions in include/pa.h."""
import math

import torch


def angles(positions, frequencies):
    """fp64 [T, R / 2]: position * frequency, whole turns dropped in Python's integers."""
    out = torch.zeros(len(positions), len(frequencies), dtype=torch.float64)
    for t, p in enumerate(positions.tolist()):
        for i, f in enumerate(frequencies.tolist()):
            turn = (p * (f % 2 ** 64)) % 2 ** 64
            if turn >= 2 ** 63:
                turn -= 2 ** 64  # in [-1/2, 1/2): the conversion below keeps 53 bits of it
            out[t, i] = turn / 2.0 ** 64 * 2.0 * math.pi
    return out


def rows(x, positions, frequencies, interleaved=False, magnitude=1.0, weight=None, eps=1e-6):
    """(values, bound): the rotated rows [T, H, D] in fp64, and how far an fp32 evaluation rounded to x's
    type may be from them.

    The bound, in units of u = 2^-24 and of m (|a| + |b|) of the pair.  Norm: the mean square is a sum of
    positive terms, 16 products and sums in a lane and at most 4 levels of lanes, a product with 1 / D, a
    sum with eps: 22 u, of which the root takes half, 11 u; the root, two products (the power of two is
    exact), 3 u.  The reciprocal root is rounded to nearest.  Together 14 u on a and b.  cos and sin: the angle is
    rounded to 24 bits within pi / 4 (0.4 u) and 31 bits of a turn (0.1 u), sincospif is within one unit
    in the last place of a value of at most 1 (2 u), the product with m 1 u: 3.5 u.  The rotation: a
    product and a fused product and sum, 2 u.  14 + 3.5 + 2 < 20 with a norm, 6 without.  Then the result is
    rounded to its type by at most half a step."""
    y = x.double().cpu()
    D = y.shape[-1]
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double().cpu()
    R = 2 * (0 if frequencies is None else len(frequencies))
    out, size = y.clone(), y.abs()
    if R:
        angle = angles(positions.cpu(), frequencies.cpu())[:, None, :]
        c, s = magnitude * torch.cos(angle), magnitude * torch.sin(angle)
        first = slice(0, R, 2) if interleaved else slice(0, R // 2)
        second = slice(1, R, 2) if interleaved else slice(R // 2, R)
        a, b = y[..., first], y[..., second]
        out[..., first] = a * c - b * s
        out[..., second] = b * c + a * s
        size[..., first] = size[..., second] = abs(magnitude) * (a.abs() + b.abs())
    u = 2.0 ** -24
    bound = (6 if weight is None else 20) * u * size
    half_step = torch.finfo(x.dtype).eps / 2
    tiny = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps / 2  # below the normal numbers
    return out, bound + half_step * (out.abs() + bound) + tiny


def assert_rows(got, want, bound, what=""):
    d = (got.double().cpu() - want).abs()
    assert bool((d <= bound).all()), "%s: %d of %d outside, worst %.3g of the bound" % (
        what, int((d > bound).sum()), d.numel(), float((d / bound).max()))
