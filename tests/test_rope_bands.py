"""MOE_ROPE_BANDS where the trained length is so short, or the bands so placed, that a band
lies before the first pair or behind the last."""
import math
import os

import numpy as np
import pytest


@pytest.fixture(scope="module")
def L():
    from routing_q4_grouped_gb300 import build, moeq4
    if not os.path.exists(moeq4.LIB_PATH):
        build.build()
    return moeq4


@pytest.mark.parametrize("rot", [2, 8, 64, 128])
@pytest.mark.parametrize("trained,fast,slow", [(4, 32, 1), (6, 2, 1), (100, 32, 1), (4096, 32, 1),
                                               (4096, 700, 690), (1e9, 32, 1), (1e12, 1e-3, 1e-4),
                                               (64, 12, 11)])
def test_bands_keep_and_divide(L, rot, trained, fast, slow):
    base, factor = 1e4, 16.0
    ph = L.moe_rope_phases(rot, base, 3, factor, trained=trained, fast=fast, slow=slow)
    got = ph.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    f = base ** (-2.0 * np.arange(rot // 2) / rot)
    turns = trained * f / (2 * math.pi)
    close = dict(rtol=1e-14, atol=2 * math.pi * 2.0 ** -64)
    stay, slowed = turns >= fast * (1 + 1e-12), turns <= slow * (1 - 1e-12)
    assert np.allclose(got[stay], f[stay], **close)
    assert np.allclose(got[slowed], f[slowed] / factor, **close)
    slack = f * close["rtol"] + close["atol"]
    assert np.all(got <= f + slack) and np.all(got >= f / factor - slack)
