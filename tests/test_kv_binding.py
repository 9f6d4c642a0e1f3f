"""The binding refuses missing tensors of the attention side by name."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from routing_q4_grouped_gb300 import build, moeq4
    if not os.path.exists(moeq4.LIB_PATH):
        build.build()
    return moeq4


def test_missing_tensors(L):
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="moe_rope: x must be"):
        L.moe_rope(None, x, None, None)
    with pytest.raises(ValueError, match="moe_kv_read: slots must be"):
        L.moe_kv_read(None, None)
