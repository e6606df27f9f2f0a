"""pa_decode_accumulate when only some of a sequence's heads set an error: the sequence adds nothing at all."""
import numpy as np
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


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 64), (64, 4, 128)])
@pytest.mark.parametrize("P", [-1, 256, pa.PA_PARTITION_BALANCED], ids=["unsplit", "p256", "balanced"])
def test_a_sequence_adds_for_all_heads_or_none(Hq, Hkv, D, P):
    """Waits that run out at once, or after a few polls (then perhaps in some units only): a sequence any of
    whose output rows was left unwritten adds nothing, and every other adds Hq / Hkv for every KV head."""
    lens = [1100, 40, 700, 16, 1, 333, 2000, 90]
    c = make_case(len(lens), Hq, Hkv, D, lens, seed=D)
    g = to_gpu(c)
    G, W = Hq // Hkv, g.block_table.shape[1] * 16
    for limit in [-1, 1, 2, 3, 4, 0] * 4:
        weights = torch.zeros(c.S, Hkv, W, device="cuda")
        g.out.fill_(float("nan"))
        pa.pa_decode_accumulate(g.out, g.q, g.k_cache, g.v_cache, g.block_table, g.seq_lens, c.scale, Hkv, weights,
                                partition_size=P, device_error=g.err, first_wait_limit=limit)
        status = pa.pa_check_device_error(g.err)
        assert status in ((0, 0), (-8, pa.PA_DEVERR_WAIT_TIMEOUT))
        wrote = ~g.out.isnan().any(-1).any(-1).cpu().numpy()
        total = weights.sum(-1).cpu().numpy()
        for s in range(c.S):
            assert np.allclose(total[s], G if wrote[s] else 0.0, atol=1e-3), (limit, s, wrote[s], total[s])
