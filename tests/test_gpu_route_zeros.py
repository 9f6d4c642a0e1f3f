"""Zeros of both signs among router logits: +0.0 and -0.0 are equal numbers, so a choice between
them goes to the lower expert."""
import numpy as np
import pytest

import oracle as O
from gpu_helpers import assert_route_equal, dev, route_gpu, route_np
from routing_q4_grouped_gb300 import moeq4
from test_gpu_route_scored import _check

pytestmark = pytest.mark.gpu


def _zeros(T, E, seed, others):
    """Rows of zeros of random signs, with a few other numbers among them."""
    rng = np.random.default_rng(seed)
    z = np.where(rng.random((T, E)) < 0.5, np.float32(-0.0), np.float32(0.0))
    at = rng.random((T, E)) < others
    return np.where(at, rng.choice(np.array([-1.0, 1.0, 1e-30, -1e-30], np.float32), (T, E)), z)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,E", [(1, 4), (7, 64), (100, 33), (40, 256), (9, 384), (5, 1000),
                                 (2100, 64)])
def test_zeros_of_both_signs(T, E, sigmoid):
    for others in (0.0, 0.1, 0.5):
        z = _zeros(T, E, T + E, others)
        _check(z, min(E, 6), sigmoid=sigmoid)
        _check(z, 1, sigmoid=sigmoid, renorm=False)
    _check(np.tile(np.array([[-0.0, 0.0, -1.0, -2.0]], np.float32), (T, 1)), 1, sigmoid=sigmoid)
    _check(np.tile(np.array([[-1.0, 0.0, -0.0, 0.0]], np.float32), (T, 1)), 2, sigmoid=sigmoid)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T", [3, 90, 2100])
@pytest.mark.parametrize("E,groups,top", [(64, 8, 3), (60, 12, 5), (256, 8, 4), (384, 6, 2)])
def test_zeros_in_groups(T, E, groups, top, sigmoid):
    if T > 1000 and E != 64:
        T = 130
    for others in (0.0, 0.02, 0.3):
        z = _zeros(T, E, T + E + groups, others)
        for best in (1, 2):
            _check(z, 5, sigmoid=sigmoid, groups=groups, top_groups=top, group_best=best)
        # a bias of zeros of both signs: keys are scores plus that
        bias = np.where(np.arange(E) % 3 == 0, np.float32(-0.0), np.float32(0.0))
        _check(z, 5, sigmoid=sigmoid, bias=bias, groups=groups, top_groups=top)


def test_zeros_beside_a_number_that_is_not_finite():
    # the row goes through the whole choice in 64 bits: the same experts
    z = _zeros(50, 64, 5, 0.05)
    z[:, 63] = -np.inf
    _check(z, 6, err=moeq4.MOE_DEVERR_NONFINITE_LOGIT)


@pytest.mark.parametrize("T,E,k", [(1, 4, 1), (7, 64, 6), (100, 33, 8), (40, 256, 8), (9, 384, 5),
                                   (5, 1000, 32), (2100, 64, 4)])
def test_plain_routing(T, E, k):
    for others in (0.0, 0.1, 0.5):
        z = _zeros(T, E, T + E, others)
        out, err, _ = route_gpu(z, k, 128)
        assert err == 0
        assert_route_equal(route_np(out), O.route(z, k, 128))


def test_router_of_rows_without_signal():
    # products of zeros: logits of either sign of zero, all equal
    rng = np.random.default_rng(9)
    x = O.to_bf16(np.where(rng.random((200, 128)) < 0.5, np.float32(-0.0), np.float32(0.0)))
    w = O.to_bf16(rng.standard_normal((64, 128)).astype(np.float32))
    out = moeq4.RouteBuffers.alloc(200, 64, 8)
    logits = dev(np.full((200, 64), 7.0, np.float32))
    moeq4.moe_router_topk(dev(x), dev(w), out, logits)
    assert moeq4.moe_get_device_error(out) == 0 and (logits == 0).all()
    assert (out.ids.cpu().numpy() == np.arange(8)).all()
