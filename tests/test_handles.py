"""Handles of calls: parts that were checked together cannot be replaced one by one, and a call
takes its pointers from the tensors as they are when it is made."""
import ctypes
import os

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from routing_q4_grouped_gb300 import build, moeq4
    if not os.path.exists(moeq4.LIB_PATH):
        build.build()
    return moeq4


@pytest.mark.parametrize("name,value", [("score", 0), ("bias", torch.zeros(8)), ("groups", 7),
                                        ("top_groups", 3), ("group_best", 2), ("renorm", False),
                                        ("factor", 2.0)])
def test_a_score_stays_as_it_was_made(L, name, value):
    s = L.RouteScore(L.MOE_SCORE_SIGMOID, groups=4, top_groups=2, factor=1.5)
    old, packed = getattr(s, name), s.packed()
    with pytest.raises(AttributeError, match=f"RouteScore: {name} cannot be replaced"):
        setattr(s, name, value)
    assert getattr(s, name) is old and s.packed() == packed


def test_packed_score_is_the_structure(L):
    s = L.RouteScore(L.MOE_SCORE_SIGMOID, None, 8, 4, 2, False, 2.5)
    assert ctypes.sizeof(L.RouteScoreC) == L._SCORE.size
    c = L.RouteScoreC.from_buffer_copy(s.packed())
    assert (c.bias, c.score, c.groups, c.top_groups, c.group_best, c.renorm, c.factor) == \
        (None, 1, 8, 4, 2, 0, 2.5)


def _route(L, z, score):
    T, E = z.shape
    out = L.RouteBuffers.alloc(T, E, 4)
    L.moe_route_scored(z, score, out, L.alloc_workspace(L.moe_route_workspace_size(T, E, 4)))
    assert L.moe_get_device_error(out) == 0
    return out.ids


@pytest.mark.gpu
def test_a_bias_moved_under_its_tensor(L):
    # the same tensor object, other memory (as moving or loading a module's parameters does)
    z = torch.randn((50, 64), device="cuda")
    old, new = (0.5 * torch.randn(64, device="cuda") for _ in range(2))
    bias = old.clone()
    score = L.RouteScore(L.MOE_SCORE_SIGMOID, bias)
    first = _route(L, z, score).clone()
    kept = bias.data                        # (the old memory stays in use, with the old values)
    bias.data = new.clone()
    assert torch.equal(_route(L, z, score), _route(L, z, L.RouteScore(L.MOE_SCORE_SIGMOID, new)))
    bias.data = kept
    assert torch.equal(_route(L, z, score), first)
    bias.data = torch.zeros(32, device="cuda")
    with pytest.raises(ValueError, match="bias must hold 64"):
        _route(L, z, score)
    bias.data = torch.zeros(128, device="cuda")[::2]
    with pytest.raises(ValueError, match="contiguous=False"):
        _route(L, z, score)


@pytest.mark.gpu
def test_values_in_place_are_seen(L):
    z = torch.randn((20, 64), device="cuda")
    bias = torch.zeros(64, device="cuda")
    score = L.RouteScore(L.MOE_SCORE_SIGMOID, bias)
    bias[7] = 10.0
    assert (_route(L, z, score)[:, 0] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["weight", "bias", "scale", "err", "N", "K", "dtype"])
def test_a_projection_stays_as_it_was_made(L, name):
    lin = L.Linear(torch.zeros((64, 128), dtype=torch.bfloat16, device="cuda"),
                   torch.zeros(64, device="cuda"))
    old = getattr(lin, name)
    with pytest.raises(AttributeError, match=f"Linear: {name} cannot be replaced"):
        setattr(lin, name, None)
    assert getattr(lin, name) is old


@pytest.mark.gpu
def test_weights_moved_under_their_tensor(L):
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").float()   # noqa: E731
    w, bias, x = rnd(40, 64).bfloat16(), rnd(40), rnd(5, 64).bfloat16()
    lin, out = L.Linear(w, bias), torch.empty((5, 40), device="cuda")
    # other memory, another row stride, another bias
    w.data = torch.cat((rnd(40, 64), rnd(40, 64)), 1).bfloat16()[:, 64:]
    bias.data = rnd(40)
    L.moe_linear(x, lin, out)
    assert torch.equal(out, x.float() @ w.float().t() + bias)
    for bad in (rnd(39, 64), rnd(40, 72), rnd(64, 40).t()):
        w.data = bad.bfloat16() if bad.is_contiguous() else bad.bfloat16().t().contiguous().t()
        with pytest.raises(ValueError, match="moe_linear: weight must be"):
            L.moe_linear(x, lin, out)
    w.data = rnd(40, 64).bfloat16()
    bias.data = rnd(39)
    with pytest.raises(ValueError, match="moe_linear: bias must hold 40"):
        L.moe_linear(x, lin, out)
    assert L.moe_get_device_error(lin) == 0
