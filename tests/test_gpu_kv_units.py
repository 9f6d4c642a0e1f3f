"""Attention over shares that cut units of different kinds in one block: row tiles of
one and two query tiles, requests of zero to many tokens, a prefix before them."""
import numpy as np
import pytest
import torch

from test_gpu_kv import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (128, 8), (256, 4)])
@pytest.mark.parametrize("nq,G,lens,prefix", [
    (20, 8, [300, 0, 19, 700, 1, 64], 0),        # 160 rows: one query tile (and a part of a second)
    (40, 8, [300, 0, 39, 500, 700], 0),          # 320 rows: units with two and with one query tile
    (9, 40, [260, 10, 515], 200),                # 360 rows per request, 1080 behind the prefix
    (3, 24, [5, 600, 0, 2], 1300),               # 72 rows per request, 288 behind the prefix
    (70, 1, [70] * 9 + [1000], 0),               # 70 rows per unit
])
def test_units_of_mixed_size(D, bits, nq, G, lens, prefix):
    c = Case(nq + G, lens, G, 1, D, bits, 48, prefix=prefix, nq=nq)
    out = c.run()
    c.check(out)
    assert np.array_equal(out.cpu().view(dtype=torch.int16).numpy(),
                          c.run().cpu().view(dtype=torch.int16).numpy())


def test_many_units_per_block():
    # 200 requests of one head: more units than blocks, so shares run through several
    lens = [(37 * b) % 300 for b in range(200)]
    c = Case(5, lens, 66, 1, 64, 8, 16, nq=1)
    c.check(c.run())
