"""Handles of calls: parts that were checked together cannot be replaced one by one, and a call
takes its pointers from the tensors as they are when it is made."""
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
    old = getattr(s, name)
    with pytest.raises(AttributeError, match=f"RouteScore: {name} cannot be replaced"):
        setattr(s, name, value)
    assert getattr(s, name) is old


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
    bias.data = torch.zeros(64)
    with pytest.raises(ValueError, match="on cpu"):
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
    bias.data = torch.zeros(40)
    with pytest.raises(ValueError, match="moe_linear: bias must hold 40 .* on cpu"):
        L.moe_linear(x, lin, out)
    w.data = torch.zeros((40, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="moe_linear: weight must be .* on cpu"):
        L.moe_linear(x, lin, out)
    assert L.moe_get_device_error(lin) == 0


ARRAYS = ["ids", "w", "counts", "offsets", "perm", "inv", "tiles", "n_tiles", "err"]


@pytest.mark.parametrize("name", ARRAYS)
def test_results_on_the_host_are_refused(L, name):
    out = L.RouteBuffers.alloc(4, 8, 2, device="cpu")
    out.check("f", -1)                      # (-1: what tensors on the host say of their device)
    with pytest.raises(ValueError, match="f: ids of the result must be"):
        out.check("f", 0)
    setattr(out, name, None)
    with pytest.raises(ValueError, match=f"f: {name} of the result must be"):
        out.check("f", -1)


@pytest.mark.parametrize("name,value", [("T", 5), ("k", 3), ("E", 9), ("block_m", 1)])
def test_results_of_other_sizes_are_refused(L, name, value):
    out = L.RouteBuffers.alloc(4, 8, 2, 128, device="cpu")
    out.check("f", -1)
    setattr(out, name, value)
    if name == "block_m":                   # tiles of 1 row: T k + min(E, T k) = 16 entries
        assert out.tiles.shape[0] < 16
    with pytest.raises(ValueError, match="of the result must be"):
        out.check("f", -1)


def test_workspaces_that_do_not_fit_are_refused(L):
    for ws in (None, torch.zeros(256, dtype=torch.uint8), torch.zeros(256)):
        with pytest.raises(ValueError, match="f: the workspace must be"):
            L._workspace("f", ws, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("scored", [False, True])
def test_routing_refuses_what_it_cannot_write(L, scored):
    T, E, k = 40, 64, 4
    z = torch.randn((T, E), device="cuda")
    size = L.moe_route_workspace_size(T, E, k)
    ws = L.alloc_workspace(size)
    score = L.RouteScore()
    call = (lambda o, w: L.moe_route_scored(z, score, o, w)) if scored else \
        (lambda o, w: L.moe_route(z, o, w))
    out = L.RouteBuffers.alloc(T, E, k)
    call(out, ws)
    want = out.ids.clone()
    for w in (None, ws.cpu(), ws.float(), ws.repeat(2)[::2]):
        with pytest.raises(ValueError, match="the workspace must be"):
            call(out, w)
    with pytest.raises(L.MoeError):
        call(out, ws[:16])
    for name in ARRAYS:
        a = getattr(out, name)
        for bad in (None, a.cpu(), a.short(), a.flatten()[:0], torch.stack((a, a), -1)[..., 0]):
            setattr(out, name, bad)
            with pytest.raises(ValueError, match=f"{name} of the result must be"):
                call(out, ws)
        setattr(out, name, a)
    for name, value in (("T", T + 1), ("k", k + 1), ("E", E + 1)):
        old = getattr(out, name)
        setattr(out, name, value)
        with pytest.raises(ValueError):
            call(out, ws)
        setattr(out, name, old)
    out.ids.zero_()
    call(out, ws)
    assert torch.equal(out.ids, want) and L.moe_get_device_error(out) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("scored", [False, True])
def test_layer_refuses_what_it_cannot_read_or_write(L, scored):
    from routing_q4_grouped_gb300 import synth
    cfg = synth.CONFIGS["tiny"]
    T = 16
    W = L.DeviceWeights.from_host(synth.gen_weights(cfg))
    x, y = (torch.zeros((T, cfg.d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    z = torch.randn((T, cfg.E), device="cuda")
    out = L.RouteBuffers.alloc(T, cfg.E, cfg.k)
    ws = L.alloc_workspace(L.moe_layer_workspace_size(T, cfg.E, cfg.k, cfg.d, cfg.f, cfg.f_s))
    score = L.RouteScore()

    def call(x=x, z=z, y=y, ws=ws, out=out):
        if scored:
            L.moe_layer_scored(x, z, W, score, out, y, ws)
        else:
            L.moe_layer(x, z, W, out, y, ws)

    call()
    for kw in (dict(ws=ws.cpu()), dict(ws=None), dict(y=y[:-1].contiguous()),
               dict(x=x[:, :64].contiguous()), dict(z=z[:-1].contiguous()), dict(z=z.cpu()),
               dict(out=L.RouteBuffers.alloc(T, cfg.E, cfg.k, device="cpu"))):
        with pytest.raises(ValueError):
            call(**kw)
    call()
    assert L.moe_get_device_error(out) == 0
    if scored:
        packed = W.packed
        for bad in (None, packed[:-256].contiguous(), packed.cpu()):
            W.packed = bad
            with pytest.raises(ValueError, match="weights"):
                call()
        W.packed = packed


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["data", "err", "pages", "page_size", "Hkv", "D", "bits"])
def test_a_cache_stays_as_it_was_made(L, name):
    cache = L.KVCache.alloc(4, 16, 2, 64, 8)
    old = getattr(cache, name)
    with pytest.raises(AttributeError, match=f"KVCache: {name} cannot be replaced"):
        setattr(cache, name, None)
    assert getattr(cache, name) is old


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["phase", "rot", "interleaved", "mscale"])
def test_rotary_positions_stay_as_they_were_made(L, name):
    rope = L.RopeSpec(L.moe_rope_phases(64, 10000.0).cuda(), 64)
    old = getattr(rope, name)
    with pytest.raises(AttributeError, match=f"RopeSpec: {name} cannot be replaced"):
        setattr(rope, name, None)
    assert getattr(rope, name) is old


@pytest.mark.gpu
@pytest.mark.parametrize("scored", [False, True])
def test_no_tokens_need_no_arrays(L, scored):
    out = L.RouteBuffers.alloc(0, 16, 2)
    ws = L.alloc_workspace(L.moe_route_workspace_size(0, 16, 2))
    z = torch.empty((0, 16), device="cuda")
    for name in ("ids", "w", "perm", "inv"):
        setattr(out, name, None)
    out.counts.fill_(5)
    if scored:
        L.moe_route_scored(z, L.RouteScore(), out, ws)
    else:
        L.moe_route(z, out, ws)
    assert L.moe_get_device_error(out) == 0
    assert (out.counts == 0).all() and (out.offsets == 0).all() and out.n_tiles[0] == 0
    out.counts = None
    with pytest.raises(ValueError, match="counts of the result must be"):
        L.moe_route(z, out, ws)


def test_packed_result_is_the_structure(L):
    for T in (0, 4):
        out = L.RouteBuffers.alloc(T, 8, 2, device="cpu")
        assert out.packed() == bytes(out.cstruct())
