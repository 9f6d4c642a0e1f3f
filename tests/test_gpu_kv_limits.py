"""Lengths against max_len = 0: nothing of a request's own is seen, and lengths other than 0
are reported."""
import pytest
import torch

from kv_case import Case
from routing_q4_grouped_gb300 import moeq4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix", [0, 70])
@pytest.mark.parametrize("B,Hq", [(3, 4), (200, 16)])
def test_lengths_with_no_room_for_any(B, Hq, prefix):
    c = Case(B, [0] * B, Hq, 2, 64, 8, 16, prefix=prefix, nq=2)
    clean = c.run()
    c.check(clean)
    for bad in (1, -1):
        c.lens[B - 1] = bad
        out = c.run()
        assert torch.equal(out, clean)
        assert moeq4.moe_get_device_error(c.cache) == moeq4.MOE_DEVERR_BAD_LENGTH
        c.cache.err.zero_()
        c.lens[B - 1] = 0
