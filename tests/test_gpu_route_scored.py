"""moe_route_scored and moe_layer_scored against the float64 oracle: the choice and every
array behind it equal, the weights within 2^-19 of their value.

The weights' bound: fp32 scores take an exponential (2 units in the last place), a sum of at
most 32 terms per lane and a tree of 5, and three more roundings: below 2 * (2 + 37 + 3) half
units for a quotient of two such numbers, 84 * 2^-25 < 2^-18.6. A kernel in 64 bits stays far
below it.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from oracle import scored
from gpu_helpers import assert_y_close, bits, dev, route_np
from routing_q4_grouped_gb300 import moeq4, synth

pytestmark = pytest.mark.gpu

WEIGHT = 2.0 ** -18.5


def _spec(sigmoid=False, bias=None, groups=1, top_groups=1, group_best=1, renorm=True, factor=1.0):
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    kind = moeq4.MOE_SCORE_SIGMOID if sigmoid else moeq4.MOE_SCORE_SOFTMAX
    return moeq4.RouteScore(kind, b, groups, top_groups, group_best, renorm, factor)


def _check(logits, k, bm=128, err=0, **how):
    logits = np.asarray(logits, np.float32)
    T, E = logits.shape
    out = moeq4.RouteBuffers.alloc(T, E, k, bm)
    ws = moeq4.alloc_workspace(moeq4.moe_route_workspace_size(T, E, k))
    ws.fill_(255)
    moeq4.moe_route_scored(dev(logits).reshape(T, E), _spec(**how), out, ws)
    assert moeq4.moe_get_device_error(out) == err
    g, r = route_np(out), scored.route_scored(logits, k, bm, **how)
    for f in ("ids", "counts", "offsets", "perm", "inv", "tiles"):
        assert np.array_equal(g[f], getattr(r, f)), f
    assert g["n_tiles"] == len(r.tiles)
    tiny = 2.0 ** -149
    assert np.all(np.abs(g["w"] - r.w) <= np.abs(r.w) * WEIGHT + tiny)
    return g


HOWS = [dict(), dict(renorm=False, factor=1.5), dict(sigmoid=True, factor=2.5),
        dict(sigmoid=True, renorm=False)]


@pytest.mark.parametrize("how", HOWS)
@pytest.mark.parametrize("T,E,k,bm", [(1, 256, 8, 128), (8, 256, 8, 128), (9, 256, 8, 64),
                                      (33, 60, 4, 16), (7, 1, 1, 1), (16, 8, 8, 128),
                                      (65, 1000, 32, 128), (2, 1024, 1, 128), (300, 33, 5, 16),
                                      (2000, 64, 6, 128)])
def test_shapes(T, E, k, bm, how):
    rng = np.random.default_rng(T * 7 + E)
    logits = 1.5 * rng.standard_normal((T, E))
    _check(logits, k, bm, **how)
    _check(logits, k, bm, bias=0.2 * rng.standard_normal(E), **how)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,groups,top,best,k", [
    (256, 8, 4, 2, 8), (256, 8, 3, 1, 8), (64, 32, 5, 2, 10), (64, 4, 1, 1, 16), (72, 12, 5, 2, 9),
    (160, 8, 3, 1, 6), (1024, 32, 1, 2, 32), (30, 3, 3, 2, 7), (32, 32, 9, 1, 9), (512, 2, 1, 2, 32),
    (96, 3, 2, 2, 8)])
def test_groups(E, groups, top, best, k, sigmoid):
    rng = np.random.default_rng(E + groups)
    for T in (3, 130):
        logits = 1.5 * rng.standard_normal((T, E))
        for bias in (None, 0.3 * rng.standard_normal(E)):
            _check(logits, k, sigmoid=sigmoid, bias=bias, groups=groups, top_groups=top,
                   group_best=best, factor=2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_equal_keys_go_to_the_lower_expert(sigmoid):
    rng = np.random.default_rng(3)
    z = rng.integers(-2, 3, (200, 64)) * 0.25
    _check(z, 6, 16, sigmoid=sigmoid)
    _check(z, 6, 16, sigmoid=sigmoid, groups=8, top_groups=3, group_best=2)
    _check(z, 6, 16, sigmoid=sigmoid, bias=np.repeat([0.5, 0.25], 32), groups=8, top_groups=5)
    _check(np.zeros((40, 32)), 32, sigmoid=sigmoid)
    _check(np.zeros((9, 32)), 4, sigmoid=sigmoid, groups=8, top_groups=2, group_best=2)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_keys_a_few_units_apart(sigmoid):
    # logits that differ in their last bits, where the fp32 scores cannot tell them apart
    rng = np.random.default_rng(4)
    one = np.float32(1.0)
    z = (one + rng.integers(0, 40, (300, 128)).astype(np.float32) * np.float32(2.0 ** -23))
    _check(z, 8, sigmoid=sigmoid)
    _check(z, 8, sigmoid=sigmoid, groups=8, top_groups=4, group_best=2)
    # keys that meet although the logits differ: the bias undoes the score up to its rounding
    z = rng.standard_normal(128).astype(np.float32)
    s = 1.0 / (1.0 + np.exp(-z.astype(np.float64))) if sigmoid else \
        np.exp(z.astype(np.float64)) / np.exp(z.astype(np.float64)).sum()
    bias = (0.75 - s).astype(np.float32)
    _check(np.tile(z, (20, 1)), 8, sigmoid=sigmoid, bias=bias, groups=4, top_groups=2, group_best=2)


@pytest.mark.parametrize("T", [4, 200])
def test_values_out_of_range(T):
    rng = np.random.default_rng(5)
    z = rng.standard_normal((T, 64))
    z[:, 3], z[:, 9], z[:, 20] = math.nan, -math.inf, math.inf
    bad = moeq4.MOE_DEVERR_NONFINITE_LOGIT
    for sigmoid in (False, True):
        _check(z, 8, err=bad, sigmoid=sigmoid)
        _check(z, 8, err=bad, sigmoid=sigmoid, groups=8, top_groups=3, group_best=2)
    _check(np.full((T, 64), math.nan), 8, err=bad)
    _check(np.full((T, 64), -math.inf), 8, err=bad, sigmoid=True)
    # scores that fp32 does not hold, and that 64 bits do not hold
    for low in (-90.0, -120.0, -300.0, -700.0, -1000.0):
        _check(low - rng.random((T, 64)), 8, sigmoid=True)
        _check(low - rng.random((T, 64)), 8, sigmoid=True, groups=8, top_groups=2, renorm=False)
    _check(3e38 * np.sign(rng.standard_normal((T, 64))), 8)
    _check(200.0 * rng.standard_normal((T, 64)), 8, groups=4, top_groups=2)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_biases_out_of_range(sigmoid):
    # experts taken out of use, one forced in, a bias that is not a number
    rng = np.random.default_rng(6)
    z = rng.standard_normal((50, 64))
    bias = 0.1 * rng.standard_normal(64)
    bias[:40] = -math.inf
    bias[50] = math.inf
    bias[51] = math.nan
    _check(z, 8, sigmoid=sigmoid, bias=bias)
    _check(z, 30, sigmoid=sigmoid, bias=bias)            # more than are left
    _check(z, 8, sigmoid=sigmoid, bias=bias, groups=8, top_groups=2, group_best=2)
    _check(z, 8, sigmoid=sigmoid, bias=bias * 1e30, groups=8, top_groups=4, group_best=2)
    _check(z, 8, sigmoid=sigmoid, bias=np.full(64, 1e7), groups=8, top_groups=4, group_best=2)


def test_no_tokens():
    out = moeq4.RouteBuffers.alloc(0, 16, 2)
    ws = moeq4.alloc_workspace(moeq4.moe_route_workspace_size(0, 16, 2))
    moeq4.moe_route_scored(torch.empty((0, 16), device="cuda"), _spec(), out, ws)
    assert moeq4.moe_get_device_error(out) == 0
    assert (out.counts == 0).all() and (out.offsets == 0).all() and out.n_tiles[0] == 0


def test_many_tokens_and_repeats():
    rng = np.random.default_rng(8)
    z = 1.5 * rng.standard_normal((20000, 256)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(256)).astype(np.float32)
    how = dict(sigmoid=True, groups=8, top_groups=4, group_best=2, factor=2.5)
    out = moeq4.RouteBuffers.alloc(20000, 256, 8)
    ws = moeq4.alloc_workspace(moeq4.moe_route_workspace_size(20000, 256, 8))
    moeq4.moe_route_scored(dev(z), _spec(bias=bias, **how), out, ws)
    first = {f: getattr(out, f).clone() for f in ("ids", "w", "perm", "inv", "counts", "offsets")}
    moeq4.moe_route_scored(dev(z), _spec(bias=bias, **how), out, ws)
    for f, v in first.items():
        assert torch.equal(v, getattr(out, f)), f
    at = rng.choice(20000, 300, replace=False)
    r = scored.route_scored(z[at], 8, bias=bias, **how)
    assert np.array_equal(out.ids.cpu().numpy()[at], r.ids)
    counts, offsets, perm, inv, tiles = scored.arrays(out.ids.cpu().numpy(), 256, 128)
    g = route_np(out)
    for f, v in dict(counts=counts, offsets=offsets, perm=perm, inv=inv, tiles=tiles).items():
        assert np.array_equal(g[f], v), f


@pytest.mark.parametrize("T", [2, 64])
def test_layer(T):
    cfg = synth.CONFIGS["tiny"]
    W = synth.gen_weights(cfg)
    x = synth.gen_x(cfg)[:T]
    logits = synth.gen_logits(cfg)[:T]
    bias = np.linspace(-0.2, 0.2, cfg.E).astype(np.float32)
    how = dict(sigmoid=True, bias=bias, groups=4, top_groups=2, group_best=1, factor=1.5)
    D = moeq4.DeviceWeights.from_host(W)
    out = moeq4.RouteBuffers.alloc(T, cfg.E, cfg.k)
    ws = moeq4.alloc_workspace(moeq4.moe_layer_workspace_size(T, cfg.E, cfg.k, cfg.d, cfg.f,
                                                             cfg.f_s, 128))
    y = torch.empty((T, cfg.d), dtype=torch.bfloat16, device="cuda")
    moeq4.moe_layer_scored(dev(x), dev(logits), D, _spec(**how), out, y, ws)
    assert moeq4.moe_get_device_error(out) == 0
    r = scored.route_scored(logits, cfg.k, **how)
    assert np.array_equal(out.ids.cpu().numpy(), r.ids)
    r.w = r.w.astype(np.float32)
    assert_y_close(bits(y), O.expert_ffn(x, W, r))


def test_captured_with_changing_logits():
    z = torch.randn((100, 64), device="cuda")
    out, ref = (moeq4.RouteBuffers.alloc(100, 64, 4) for _ in range(2))
    ws = moeq4.alloc_workspace(moeq4.moe_route_workspace_size(100, 64, 4))
    spec = _spec(sigmoid=True, groups=8, top_groups=2, group_best=2)
    moeq4.moe_route_scored(z, spec, out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moeq4.moe_route_scored(z, spec, out, ws)
    for i in range(3):
        z.normal_()
        g.replay()
        moeq4.moe_route_scored(z, spec, ref, ws)
        for f in ("ids", "w", "perm", "inv", "counts", "offsets"):
            assert torch.equal(getattr(out, f), getattr(ref, f)), (i, f)


def test_binding_refusals():
    out = moeq4.RouteBuffers.alloc(4, 64, 4)
    ws = moeq4.alloc_workspace(moeq4.moe_route_workspace_size(4, 64, 4))
    with pytest.raises(ValueError, match="logits must be"):
        moeq4.moe_route_scored(torch.zeros((4, 32), device="cuda"), _spec(), out, ws)
    with pytest.raises(ValueError, match="bias must hold"):
        moeq4.moe_route_scored(torch.zeros((4, 64), device="cuda"), _spec(bias=np.zeros(32)), out, ws)
    with pytest.raises(moeq4.MoeError):
        moeq4.moe_route_scored(torch.zeros((4, 64), device="cuda"), _spec(groups=7), out, ws)


@pytest.mark.parametrize("E,groups,best", [(256, 8, 2), (64, 8, 1), (128, 4, 2), (60, 12, 2)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_keys_near_the_rounding_of_fp32(E, groups, best, sigmoid):
    # distances between keys from far below to above what fp32 scores resolve, within a lane's
    # experts and across them, at the border of the choice and of the groups
    rng = np.random.default_rng(E + best)
    base = rng.standard_normal(E)
    for step in (2.0 ** -24, 2.0 ** -22, 2.0 ** -20, 2.0 ** -18, 2.0 ** -16, 2.0 ** -12):
        z = (rng.choice(base[:6], (60, E)) + step * rng.integers(-3, 4, (60, E)))
        for bias in (None, 0.25 + step * rng.integers(-2, 3, E)):
            _check(z, 6, sigmoid=sigmoid, bias=bias)
            _check(z, 6, sigmoid=sigmoid, bias=bias, groups=groups, top_groups=groups // 2,
                   group_best=best, renorm=False)
            _check(z, 6, sigmoid=sigmoid, bias=bias, groups=groups, top_groups=groups,
                   group_best=best)


@pytest.mark.parametrize("top", [14.9, 16.0, 20.0, 30.0, 40.0])
def test_saturated_scores(top):
    # sigmoids that round to the same number in 64 bits although the logits differ
    rng = np.random.default_rng(int(top))
    z = top + 1e-5 * rng.integers(-2, 3, (80, 64)) - (rng.random((80, 64)) < 0.8) * rng.random((80, 64)) * 8
    _check(z, 8, sigmoid=True)
    _check(z, 8, sigmoid=True, groups=8, top_groups=4)
    _check(z, 8)
    tiny = rng.standard_normal((40, 64)) * 10.0 ** rng.integers(-44, -8, (40, 64)).astype(float)
    _check(tiny, 8, sigmoid=True)
    _check(tiny, 8)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_experts_forced_in(sigmoid):
    # several +inf biases in several groups: ranks beyond fp32, equal keys
    rng = np.random.default_rng(12)
    z = rng.standard_normal((40, 64))
    for forced in ([3], [3, 5], [3, 5, 9, 11, 20], list(range(0, 64, 3)), list(range(64))):
        bias = 0.1 * rng.standard_normal(64)
        bias[forced] = math.inf
        bias[60:] = -math.inf
        for top, best in ((2, 2), (4, 2), (3, 1)):
            _check(z, 8, sigmoid=sigmoid, bias=bias, groups=8, top_groups=top, group_best=best)


@pytest.mark.parametrize("E,groups", [(300, 12), (384, 8), (384, 6), (512, 8), (640, 20), (257, 1)])
def test_more_experts(E, groups):
    rng = np.random.default_rng(E)
    for T in (5, 2100):
        z = 1.5 * rng.standard_normal((T, E))
        bias = 0.1 * rng.standard_normal(E)
        top = max(1, groups // 2)
        if T > 1000:
            z = z[rng.integers(0, 40, T)]          # (few different tokens: the oracle is slow)
        _check(z, 10, sigmoid=True, bias=bias, groups=groups, top_groups=top, group_best=2)
        _check(z, 10, renorm=False, groups=groups, top_groups=top)
