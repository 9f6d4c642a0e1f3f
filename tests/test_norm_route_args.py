"""Refusals of moe_rms_norm, moe_route_scored and moe_layer_scored: on the host, before
anything is enqueued, by the library and by the binding."""
import ctypes
import os

import pytest
import torch

FAKE = 1 << 20      # aligned, never dereferenced
ARG, SHAPE, WORKSPACE, ALIGN = -1, -2, -3, -7


@pytest.fixture(scope="module")
def L():
    from routing_q4_grouped_gb300 import build, moeq4
    if not os.path.exists(moeq4.LIB_PATH):
        build.build()
    return moeq4


def _norm(L, **kw):
    a = L.NormC()
    a.x, a.x_row, a.x_head = FAKE, 256, 128
    a.out, a.out_row, a.out_head = 2 * FAKE, 256, 128
    a.T, a.H, a.D, a.dtype, a.eps = 4, 2, 128, L.MOE_BF16, 1e-6
    for n, v in kw.items():
        setattr(a, n, v)
    return L.lib().moe_rms_norm(ctypes.byref(a), None)


@pytest.mark.parametrize("status,kw", [
    (ARG, dict(T=-1)), (ARG, dict(H=0)), (ARG, dict(D=0)), (ARG, dict(dtype=3)),
    (ARG, dict(dtype=-1)), (ARG, dict(eps=0.0)), (ARG, dict(eps=float("nan"))),
    (ARG, dict(eps=float("inf"))), (ARG, dict(offset=float("inf"))), (ARG, dict(x=None)),
    (ARG, dict(out=None)),                                          # nothing to write
    (ARG, dict(codes=3 * FAKE, codes_row=256, codes_head=128)),     # codes without scales
    (SHAPE, dict(D=16385)), (SHAPE, dict(H=65536)), (SHAPE, dict(T=1 << 30, H=2)),
    (SHAPE, dict(x_row=-1)), (SHAPE, dict(add=3 * FAKE, add_row=-256)),
    (SHAPE, dict(out_row=255)),                                     # rows of the result overlap
    (SHAPE, dict(out_head=64)),
    (SHAPE, dict(sum=3 * FAKE, sum_row=0, sum_head=128)),
    (ARG, dict(sum=2 * FAKE, sum_row=256, sum_head=128)),           # two results in one place
    (ARG, dict(out=FAKE, out_row=512)),                             # in place, other strides
    (ARG, dict(add=2 * FAKE, add_row=512, add_head=128)),
    (ARG, dict(codes=FAKE, codes_row=256, codes_head=128, scales=4 * FAKE)),   # codes over x
    (ALIGN, dict(x=FAKE + 1)), (ALIGN, dict(weight=FAKE + 1)),
    (ALIGN, dict(codes=3 * FAKE, codes_row=256, codes_head=128, scales=FAKE + 2)),
])
def test_norm_refusals(L, status, kw):
    assert _norm(L, **kw) == status


def test_norm_of_no_tokens_is_nothing(L):
    assert _norm(L, T=0, x=None, out=None) == 0
    assert L.lib().moe_rms_norm(None, None) == ARG


def _route(L, **kw):
    r = L.RouteOutC()
    for f in ("ids", "w", "counts", "offsets", "perm", "inv", "tiles", "n_tiles", "err"):
        setattr(r, f, FAKE)
    r.T, r.E, r.k, r.block_m = 16, 64, 8, 128
    s = L.RouteScoreC(None, L.MOE_SCORE_SIGMOID, 8, 4, 2, 1, 2.5)
    for n, v in kw.items():
        setattr(r if hasattr(r, n) else s, n, v)
    return r, s


@pytest.mark.parametrize("status,kw", [
    (ARG, dict(score=2)), (ARG, dict(score=-1)), (ARG, dict(renorm=2)), (ARG, dict(groups=0)),
    (ARG, dict(top_groups=0)), (ARG, dict(top_groups=9)), (ARG, dict(group_best=0)),
    (ARG, dict(group_best=3)), (ARG, dict(factor=float("nan"))), (ARG, dict(k=65)),
    (SHAPE, dict(groups=7)),                       # does not divide E
    (SHAPE, dict(groups=64, group_best=1)),        # more than 32 groups
    (SHAPE, dict(groups=32, top_groups=3)),        # k above the experts of the groups that stay
    (SHAPE, dict(E=32, groups=32, top_groups=32)),                # two best of one
    (ALIGN, dict(bias=FAKE + 2)),
])
def test_route_refusals(L, status, kw):
    r, s = _route(L, **kw)
    lib = L.lib()
    assert lib.moe_route_scored(FAKE, ctypes.byref(s), ctypes.byref(r), FAKE, 1 << 30, None) == status
    P = L.Q4PackedC(FAKE, r.E, 256, 128, 0)
    assert lib.moe_layer_scored(FAKE, FAKE, 16, ctypes.byref(P), ctypes.byref(s), ctypes.byref(r),
                                FAKE, FAKE, 1 << 40, None) == status


def test_route_pointers_and_workspace(L):
    lib = L.lib()
    r, s = _route(L)
    rp, sp = ctypes.byref(r), ctypes.byref(s)
    assert lib.moe_route_scored(FAKE, None, rp, FAKE, 1 << 30, None) == ARG
    assert lib.moe_route_scored(FAKE, sp, None, FAKE, 1 << 30, None) == ARG
    assert lib.moe_route_scored(None, sp, rp, FAKE, 1 << 30, None) == ARG
    assert lib.moe_route_scored(FAKE + 4, sp, rp, FAKE, 1 << 30, None) == ALIGN
    assert lib.moe_route_scored(FAKE, sp, rp, FAKE, 16, None) == WORKSPACE
    P = L.Q4PackedC(FAKE, 64, 256, 128, 0)
    assert lib.moe_layer_scored(FAKE, FAKE, 15, ctypes.byref(P), sp, rp, FAKE, FAKE, 1 << 40,
                                None) == SHAPE
    assert lib.moe_layer_scored(FAKE, FAKE, 16, ctypes.byref(P), sp, rp, FAKE, FAKE, 16,
                                None) == WORKSPACE
    assert lib.moe_layer_scored(FAKE, FAKE, 16, ctypes.byref(P), None, rp, FAKE, FAKE, 1 << 40,
                                None) == ARG


def test_binding_refuses_host_tensors(L):
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="moe_rms_norm: x must be"):
        L.moe_rms_norm(x, out=x)
    with pytest.raises(ValueError, match="moe_rms_norm: x must be"):
        L.moe_rms_norm(None)
    with pytest.raises(ValueError, match="moe_rms_norm: x must be"):
        L.moe_rms_norm(x.to(torch.int32))
    with pytest.raises(ValueError, match="RouteScore: bias must be"):
        L.RouteScore(bias=torch.zeros(8))
    assert L.NormC.__dict__["_fields_"] and ctypes.sizeof(L.NormC) == L._NORM.size
