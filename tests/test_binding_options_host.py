"""The binding's packed options: what a caller gives is read anew in every call, in any form that int() takes."""
import numpy as np
import pytest
import torch

import paged_decode_attention_reshape_gb300 as pa


def packed(partition_size):
    return pa._decode_options(None, None, 0, None, partition_size, None, None, 0)


def want(n):
    return pa._DECODE_OPTIONS.pack(0, 0, 0, 0, n, 0, 0, 0, 0)


@pytest.mark.parametrize("form", [int, np.int64, np.array, torch.tensor, float])
def test_forms_of_a_partition_size(form):
    for n in (0, -1, 64, pa.PA_PARTITION_BALANCED, 64):
        assert packed(form(n)) == want(n)


@pytest.mark.parametrize("box", [np.array, torch.tensor])
def test_a_changed_value_is_seen(box):
    n = box(64)
    assert packed(n) == want(64)
    n += 32
    assert packed(n) == want(96)
