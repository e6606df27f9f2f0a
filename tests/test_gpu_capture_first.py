"""Calls that are captured before any eager one made the library-held workspace large enough: the
capture takes them, the workspace grows beside it, and replays, eager calls and later captures of
larger shapes give the reference's outputs.  Each case runs in a process of its own, whose workspace
is empty at the start."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PREFIX = """
import sys
sys.path[:0] = [%r, %r]
import numpy as np, torch
import fp4_cases
from gpu_cases import assert_close, make_case, reference, to_gpu
import paged_decode_attention_reshape_gb300 as pa


def case(S, Hq, Hkv, D, lens, seed):
    c = make_case(S, Hq, Hkv, D, lens, seed=seed)
    return c, to_gpu(c), reference(c)


def args(c, g):
    return (g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, c.Hkv)


def capture(call):
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        call()
    return graph


def replay(graph, c, g, ref, what):
    for it in range(2):
        g.out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        assert pa.pa_check_device_error(g.err) == (0, 0)
        assert_close(g.out.double().cpu().numpy(), ref, "%%s, replay %%d" %% (what, it))


small, big = case(2, 8, 2, 64, [500, 900], 1), case(3, 32, 8, 128, [3000, 700, 1500], 2)
""" % (ROOT, os.path.dirname(os.path.abspath(__file__)))

DECODE = """
graphs = []
for n, (c, g, ref) in enumerate((small, big)):       # the second capture grows what the first one holds
    graphs.append(capture(lambda: pa.pa_decode_opt(*args(c, g), partition_size=64, device_error=g.err)))
for n, (c, g, ref) in enumerate((small, big)):
    replay(graphs[n], c, g, ref, "graph %d" % n)
    g.out.fill_(float("nan"))
    pa.pa_decode_opt(*args(c, g), partition_size=32, device_error=g.err)      # eager, growing it again
    assert pa.pa_check_device_error(g.err) == (0, 0)
    assert_close(g.out.double().cpu().numpy(), ref, "eager %d" % n)
for n, (c, g, ref) in enumerate((small, big)):
    replay(graphs[n], c, g, ref, "graph %d again" % n)
"""

AFTER_EAGER = """
c, g, ref = small
pa.pa_decode_opt(*args(c, g), partition_size=64, device_error=g.err)
C, G, REF = big
graph = capture(lambda: pa.pa_decode_opt(*args(C, G), partition_size=64, device_error=G.err))
replay(graph, C, G, REF, "graph")
pa.pa_decode_opt(*args(C, G), partition_size=16, device_error=G.err)          # frees what the capture replaced
assert pa.pa_check_device_error(G.err) == (0, 0)
assert_close(G.out.double().cpu().numpy(), REF, "eager")
replay(graph, C, G, REF, "graph again")
"""

STEP = """
c, g, ref = big
new = [torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
slots = torch.empty(3, dtype=torch.int64, device="cuda")
for s, L in enumerate(c.lens):                       # the rows the cache holds already, written again
    blk, off = int(g.block_table[s, (L - 1) // 16]), (L - 1) % 16
    new[0][s], new[1][s], slots[s] = g.k_cache[blk, :, off], g.v_cache[blk, :, off], blk * 16 + off
graph = capture(lambda: pa.pa_decode_step(g.out, g.q, new[0], new[1], g.k_cache, g.v_cache, slots, g.block_table,
                                          g.seq_lens, c.scale, 8, partition_size=64, device_error=g.err))
replay(graph, c, g, ref, "step")
"""

ACCUMULATE = """
c, g, ref = small
weights = torch.zeros(2, 2, g.block_table.shape[1] * 16, device="cuda")
graph = capture(lambda: pa.pa_decode_accumulate(*args(c, g), weights, device_error=g.err))
replay(graph, c, g, ref, "accumulate")
total = weights.sum(-1).cpu().numpy()
assert np.allclose(total, 2 * 4, atol=1e-3), total   # two replays, 4 query heads a KV head
"""


@pytest.mark.parametrize("body", [DECODE, AFTER_EAGER, STEP, ACCUMULATE],
                         ids=["decode", "after_eager", "step", "accumulate"])
def test_captured_first(body):
    r = subprocess.run([sys.executable, "-c", PREFIX + body], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
