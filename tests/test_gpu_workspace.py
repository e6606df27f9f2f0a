"""The library-held split-KV workspace (pa_decode, and the _opt entry points without a caller
workspace): calls of different shapes share it one after another, and a captured call keeps
working when later calls make it grow."""
import pytest
import torch

from gpu_cases import assert_close, make_case, reference, to_gpu

import paged_decode_attention_reshape_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    pa.lib()
    torch.cuda.set_device(0)


def _run(c, g, P):
    g.out.fill_(float("nan"))
    pa.pa_decode_opt(g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, c.Hkv,
                     partition_size=P, device_error=g.err)
    assert pa.pa_check_device_error(g.err) == (0, 0)
    return g.out.double().cpu().numpy()


def test_calls_of_different_shapes_share_it():
    """Few units with many partial states, then many units: the second call's arrival counters
    must not be where the first call left its states (and back again)."""
    few = make_case(1, 8, 1, 64, [4000], seed=31)
    many = make_case(40, 32, 8, 64, [100 + 7 * i for i in range(40)], seed=32)
    on = [(c, to_gpu(c), reference(c)) for c in (few, many)]
    for i in (0, 1, 0, 1, 1, 0):
        c, g, ref = on[i]
        assert_close(_run(c, g, 64), ref, "shape %d" % i)


def test_captured_call_survives_growth():
    c = make_case(2, 8, 2, 64, [500, 900], seed=33)
    g, ref = to_gpu(c), reference(c)
    args = (g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, c.Hkv)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        pa.pa_decode_opt(*args, partition_size=64)      # the workspace is there before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pa.pa_decode_opt(*args, partition_size=64)
    big = make_case(3, 64, 8, 128, [9000, 8000, 700], seed=34)
    gb = to_gpu(big)
    assert_close(_run(big, gb, 64), reference(big), "the larger call")
    for it in range(2):
        g.out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert_close(g.out.double().cpu().numpy(), ref, "replay %d" % it)
