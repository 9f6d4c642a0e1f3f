"""Routing of batches whose blocks fill the shared memory that a launch may ask for: the rows of a
block's tokens grow with the batch until there is no room, then the blocks grow in number.

(experts, choices, tokens): the tokens of a block come to 136, 192 or 408, and its dynamic shared
memory to 49136 bytes, 16 below 48 KB."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_helpers import assert_route_equal, dev, route_gpu, route_np
from oracle import scored
from routing_q4_grouped_gb300 import moeq4

pytestmark = pytest.mark.gpu

SIZES = [(72, 24, 17000), (72, 17, 24000), (72, 8, 52500), (72, 8, 200000), (160, 1, 410000)]


@pytest.mark.parametrize("E,k,T", SIZES)
def test_plain_routing(E, k, T):
    z = np.random.default_rng(T).standard_normal((T, E)).astype(np.float32)
    out, err, _ = route_gpu(z, k, 128)
    assert err == 0
    assert_route_equal(route_np(out), O.route(z, k, 128))


@pytest.mark.parametrize("E,k,T", SIZES)
def test_routing_by_scores(E, k, T):
    rng = np.random.default_rng(T)
    rows = (1.5 * rng.standard_normal((50, E))).astype(np.float32)
    at = rng.integers(0, 50, T)
    out = moeq4.RouteBuffers.alloc(T, E, k)
    ws = moeq4.alloc_workspace(moeq4.moe_route_workspace_size(T, E, k))
    moeq4.moe_route_scored(dev(rows[at]), moeq4.RouteScore(moeq4.MOE_SCORE_SIGMOID), out, ws)
    assert moeq4.moe_get_device_error(out) == 0
    r = scored.route_scored(rows, k, sigmoid=True)
    counts, offsets, perm, inv, tiles = scored.arrays(r.ids[at], E, 128)
    g = route_np(out)
    assert np.array_equal(g["ids"], r.ids[at])
    assert np.all(np.abs(g["w"] - r.w[at]) <= r.w[at] * 2.0 ** -18.5)
    for f, v in dict(counts=counts, offsets=offsets, perm=perm, inv=inv, tiles=tiles).items():
        assert np.array_equal(g[f], v), f


def test_given_choice():
    # moe_route_ids: the same blocks
    T, E, k = 52500, 72, 8
    ids = np.argsort(np.random.default_rng(1).random((T, E)), axis=1)[:, :k].astype(np.int32)
    out = moeq4.RouteBuffers.alloc(T, E, k)
    out.ids.copy_(torch.from_numpy(ids))
    out.w.fill_(1.0 / k)
    ws = moeq4.alloc_workspace(moeq4.moe_route_workspace_size(T, E, k))
    moeq4.moe_route_ids(out, ws)
    assert moeq4.moe_get_device_error(out) == 0
    g = route_np(out)
    counts, offsets, perm, inv, tiles = scored.arrays(ids, E, 128)
    for f, v in dict(counts=counts, offsets=offsets, perm=perm, inv=inv, tiles=tiles).items():
        assert np.array_equal(g[f], v), f
