"""pa_decode_step refuses what its decode would refuse before the cache write is launched."""
import pytest
import torch

from gpu_cases import make_case, to_gpu

import paged_decode_attention_reshape_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    pa.lib()
    torch.cuda.set_device(0)


def refused(c, k_cache, v_cache, g, table, status, P=0):
    """The step returns `status` and leaves the caches as they were, with and without new_rows_start."""
    new = torch.ones(c.S, c.Hkv, c.D, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(c.S, device="cuda") * 16
    before = [x.view(torch.int16).clone() for x in (k_cache, v_cache)]
    for start in (None, torch.arange(c.S + 1, dtype=torch.int32, device="cuda")):
        with pytest.raises(pa.PAError) as e:
            pa.pa_decode_step(g.out, g.q, new, new, k_cache, v_cache, slots, table, g.seq_lens, c.scale, c.Hkv,
                              new_rows_start=start, partition_size=P, device_error=g.err)
        assert e.value.status == status
        torch.cuda.synchronize()
        for x, was in zip((k_cache, v_cache), before):
            assert torch.equal(x.view(torch.int16), was)


def test_workspace_that_cannot_be_had():
    """Partitions of 16 tokens over tables of 2^21 blocks: some 10^13 bytes of states."""
    c = make_case(64, 64, 8, 128, [20] * 64, seed=1)
    g = to_gpu(c)
    table = torch.zeros(64, 1 << 21, dtype=torch.int32, device="cuda")
    assert pa.pa_decode_workspace_size(64, 64, 8, 128, 1 << 21, 16) > 1 << 42
    refused(c, g.k_cache, g.v_cache, g, table, -5, 16)


@pytest.mark.parametrize("P", [0, -1, 16])
def test_caches_in_different_layouts(P):
    """K head-major and V token-major within a block: the decode takes one layout for both."""
    c = make_case(3, 8, 4, 64, [40, 17, 100], seed=2)
    g = to_gpu(c)
    v_nhd = g.v_cache.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    refused(c, g.k_cache, v_nhd, g, g.block_table, -1, P)
