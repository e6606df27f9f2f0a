"""pa_evict's refusals and pa_bm_truncate (host only; no kernel is launched here)."""
import ctypes

import pytest

from test_abi import _t

import paged_decode_attention_reshape_gb300 as pa


@pytest.fixture(scope="module")
def L():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    return pa.lib()


def _args(**over):
    S, H, D, NB, MB, B = 3, 2, 64, 16, 4, 20
    a = dict(k=_t([NB, H, 16, D], pa.PA_BF16), v=_t([NB, H, 16, D], pa.PA_BF16), bt=_t([S, MB], pa.PA_I32),
             sl=_t([S], pa.PA_I32), w=_t([S, H, MB * 16], pa.PA_F32), budget=B, recent=4,
             kept=_t([S, H, B], pa.PA_I32, ptr=0x20000), nl=_t([S], pa.PA_I32, ptr=0x30000),
             nw=_t([S, H, MB * 16], pa.PA_F32, ptr=0x40000))
    a.update(over)
    return a


def _evict(L, **over):
    a = _args(**over)
    r = [ctypes.byref(a[n]) for n in ("k", "v", "bt", "sl", "w")]
    o = [ctypes.byref(a[n]) for n in ("kept", "nl", "nw")]
    return L.pa_evict(*r, a["budget"], a["recent"], *o, None, None)


def test_refusals(L):
    S, H, D, NB, MB, B = 3, 2, 64, 16, 4, 20
    I, F = pa.PA_I32, pa.PA_F32
    assert _evict(L, budget=0) == -1
    assert _evict(L, recent=-1) == -1
    assert _evict(L, budget=21) == -1                                        # kept is [S, H, 20]
    assert _evict(L, bt=_t([S, MB], pa.PA_I64)) == -2
    assert _evict(L, sl=_t([S], pa.PA_I64)) == -2
    assert _evict(L, w=_t([S, H, MB * 16], pa.PA_BF16)) == -2
    assert _evict(L, kept=_t([S, H, B], pa.PA_I64)) == -2
    assert _evict(L, sl=_t([S + 1], I)) == -1
    assert _evict(L, bt=_t([S + 1, MB], I)) == -1
    assert _evict(L, w=_t([S, H + 1, MB * 16], F)) == -1
    assert _evict(L, w=_t([S, H, MB * 16 - 1], F), nw=_t([S, H, MB * 16 - 1], F, ptr=0x40000)) == -1
    assert _evict(L, nw=_t([S, H, MB * 16 + 1], F, ptr=0x40000)) == -1
    assert _evict(L, nw=_t([S, H, MB * 16], F)) == -1                        # the memory of weights
    assert _evict(L, nl=_t([S], I)) == -1                                    # the memory of seq_lens
    assert _evict(L, kept=_t([S, H, B], I, ptr=0)) == -1
    assert _evict(L, kept=_t([S, H, B], I, strides=[H * B * 2, B * 2, 2])) == -1
    assert _evict(L, k=_t([NB, H, 8, D], pa.PA_BF16), v=_t([NB, H, 8, D], pa.PA_BF16)) == -7
    assert _evict(L, v=_t([NB, H, 16, D], pa.PA_F16)) == -1
    assert _evict(L, k=_t([NB, H, 16, D], I), v=_t([NB, H, 16, D], I)) == -2
    assert _evict(L, k=_t([NB, H, 16, D], pa.PA_BF16, ptr=0x10008)) == -3
    big = _t([NB, H, 16, 1028], F)                                           # rows above 4096 bytes
    assert _evict(L, k=big, v=big) == -7
    page = _t([NB, H, 9 * 96], pa.PA_FP4_E2M1)
    assert _evict(L, k=page, v=page) == -7
    assert _evict(L, budget=(1 << 30) + 1, kept=_t([S, H, (1 << 30) + 1], I, ptr=0x20000)) == -7
    none = dict(bt=_t([0, MB], I), sl=_t([0], I), w=_t([0, H, MB * 16], F), kept=_t([0, H, B], I),
                nl=_t([0], I), nw=_t([0, H, MB * 16], F))
    assert _evict(L, **none) == 0                                            # an empty batch


def test_truncate(L):
    m = pa.BlockManager(8, 3, 8)
    m.append(0, 70)                      # 5 blocks
    assert m.num_free() == 3
    m.truncate(0, 33)                    # 3 blocks stay
    assert m.num_free() == 5 and m.seq_len(0) == 33
    slots, copy = m.append(0, 1)         # goes on in the block that stayed
    assert copy is None and slots[0] % 16 == 1 and m.num_free() == 5
    m.fork(0, 1)
    m.truncate(1, 16)                    # shared blocks stay with the other sequence
    assert m.num_free() == 5 and m.seq_len(1) == 16 and m.seq_len(0) == 34
    bt, sl = m.export([0, 1])
    assert bt[0, 0] == bt[1, 0] and bt[1, 1] == -1 and sl.tolist() == [34, 16]
    assert m.refs(int(bt[0, 0])) == 2 and m.refs(int(bt[0, 2])) == 1
    m.truncate(1, 0)
    assert m.seq_len(1) == 0 and m.refs(int(bt[0, 0])) == 1
    slots, _ = m.append(1, 2)            # still live
    assert m.seq_len(1) == 2
    for seq, n in ((0, 35), (0, -1), (2, 0), (7, 0), (-1, 0)):
        with pytest.raises(pa.PAError):
            m.truncate(seq, n)
    assert m.seq_len(0) == 34
