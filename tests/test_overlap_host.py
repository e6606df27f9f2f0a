"""The overlap check of pa_rotary and pa_rotary_and_cache (rows_shared in pa_validate.h), as it is compiled:
every pair of small layouts against the rows' own bytes, and the calls' refusals for views whose heads are
the outer dimension."""
import itertools
import os
import random
import subprocess

import pytest

import paged_decode_attention_reshape_gb300 as pa
from test_abi import _t
from test_rotary_host import B16, D, HKV, HQ, T, _args, _call, L  # noqa: F401  (L: the library)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D0, EB = 8, 2  # elements of a row and their bytes, in the compiled program
MAIN = r"""
#include <cstdio>
#include "pa_validate.h"
int main() {
  long long v[10];
  while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6, v + 7, v + 8, v + 9) == 10) {
    pa_tensor t[2] = {};
    for (int i = 0; i < 2; ++i) {
      t[i].data = reinterpret_cast<void *>(1000000 + v[5 * i] * %EB%);
      t[i].dtype = PA_BF16;
      t[i].ndim = 3;
      t[i].shape[0] = v[5 * i + 1], t[i].shape[1] = v[5 * i + 2], t[i].shape[2] = %D%;
      t[i].stride[0] = v[5 * i + 3], t[i].stride[1] = v[5 * i + 4], t[i].stride[2] = 1;
    }
    const bool broken = pa::rows_overlap(&t[1], %D%);
    printf("%d %d\n", broken ? 1 : 0, !broken && pa::rows_shared(&t[0], &t[1], %EB%) ? 1 : 0);
  }
}
"""


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    at = tmp_path_factory.mktemp("overlap")
    (at / "main.cpp").write_text(MAIN.replace("%EB%", str(EB)).replace("%D%", str(D0)))
    exe = str(at / "main")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", os.path.join(cuda, "include"), "-I", os.path.join(ROOT, "include"),
                           "-I", os.path.join(ROOT, "paged_decode_attention_reshape_gb300", "csrc"), str(at / "main.cpp"), "-o", exe])

    def check(pairs):  # [(x, out)], each (start, T, H, token stride, head stride) in elements
        text = "".join("%d %d %d %d %d %d %d %d %d %d\n" % (*x, *y) for x, y in pairs)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
        assert len(out) == 2 * len(pairs)
        return [(a == "1", b == "1") for a, b in zip(out[::2], out[1::2])]
    return check


def elements(v):
    start, n, h, ts, hs = v
    return {start + t * ts + i * hs + d for t in range(n) for i in range(h) for d in range(D0)}


def compare(compiled, pairs):
    """The check against the elements themselves, for outputs whose rows do not overlap one another (those are
    refused before)."""
    seen = [0, 0]
    for (x, y), (broken, got) in zip(pairs, compiled(pairs)):
        assert broken or len(elements(y)) == y[1] * y[2] * D0, y
        if not broken:
            want = bool(elements(x) & elements(y))
            assert got == want, (x, y)
            seen[want] += 1
    assert min(seen) > 100  # (both answers)


def test_views_of_equal_strides(compiled):
    """Heads inside tokens, tokens inside heads, padded or not, other numbers of heads, at every distance."""
    pairs = []
    for n in (1, 3):
        for ts, hs in ((32, 8), (40, 8), (48, 16), (8, 24), (8, 32), (16, 48), (16, 64), (24, 8), (8, 8)):
            for hx, hy in itertools.product((1, 2, 4), repeat=2):
                far = 4 * max(ts, hs) + 12
                pairs += [((5000, n, hx, ts, hs), (5000 + off, n, hy, ts, hs)) for off in range(-far, far, 3)]
    compare(compiled, pairs)


def test_views_of_other_strides(compiled):
    """A contiguous output over strided views of its buffer, transposed ones, broadcast inputs."""
    rng = random.Random(1)
    strides = (0, 4, 8, 16, 24, 32, 40, 64, 96)
    pairs = []
    for _ in range(60000):
        n = rng.choice((1, 2, 3, 5))
        x = (5000, n, rng.choice((1, 2, 3)), rng.choice(strides), rng.choice(strides))
        y = (5000 + rng.randrange(-250, 250), n, rng.choice((1, 2, 4)), rng.choice(strides), rng.choice(strides))
        pairs.append((x, y))
    compare(compiled, pairs)


OUTER = [D, T * D, 1]  # [H, T, D] buffers as [T, H, D] views


@pytest.mark.parametrize("cached", [False, True])
@pytest.mark.parametrize("rows", [T, -T, T + 1, -T - 1, 1, -1, (HQ - 1) * T, 2 * T - 1])
def test_refused_with_heads_outermost(L, cached, rows):  # noqa: F811
    a = _args(cached)
    a["q"] = _t([T, HQ, D], B16, 0x200000, strides=OUTER)
    a["q_out"] = _t([T, HQ, D], B16, 0x200000 + rows * D * 2, strides=OUTER)
    assert _call(L, a) == -1


def test_refused_with_heads_outermost_across_tensors(L):  # noqa: F811
    a = _args(False)
    a["q"], a["key"] = [_t([T, h, D], B16, 0x200000 + at * D * 2, strides=OUTER) for h, at in ((HQ, 0), (HKV, HQ * T))]
    a["q_out"] = _t([T, HQ, D], B16, a["key"].data + (T + 2) * D * 2, strides=OUTER)  # over the keys' second head
    assert _call(L, a) == -1
    a["q_out"] = _t([T, HQ, D], B16, 0x400000, strides=OUTER)
    a["k_out"] = _t([T, HKV, D], B16, 0x400000 + (HQ - 1) * T * D * 2, strides=OUTER)  # over the queries' last head
    assert _call(L, a) == -1


@pytest.mark.parametrize("cached", [False, True])
def test_refused_with_other_strides(L, cached):  # noqa: F811
    """A contiguous output over a strided view of one buffer."""
    a = _args(cached)
    a["q"] = _t([T, HQ, D], B16, 0x200000, strides=[(HQ + 2 * HKV) * D, D, 1])
    for at in (0, D * 2, 2 * HQ * D * 2, -HQ * D * 2):
        a["q_out"] = _t([T, HQ, D], B16, 0x200000 + at)
        assert _call(L, a) == -1
    a["q"] = _t([T, HQ, D], B16, 0x200000, strides=[0, D, 1])  # one token's rows for every position
    a["q_out"] = _t([T, HQ, D], B16, 0x200000 - (T - 1) * HQ * D * 2)
    assert _call(L, a) == -1
