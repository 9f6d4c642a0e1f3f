"""moe_linear on the host: refusals before anything is enqueued, and the layout of calls."""
import ctypes
import os

import pytest
import torch

FAKE = 1 << 20      # aligned, never dereferenced
ARG, SHAPE, ALIGN = -1, -2, -7


@pytest.fixture(scope="module")
def L():
    from routing_q4_grouped_gb300 import build, moeq4
    if not os.path.exists(moeq4.LIB_PATH):
        build.build()
    return moeq4


def _call(L, **kw):
    a = L.LinearC()
    a.x, a.x_row, a.w, a.w_row = FAKE, 256, 2 * FAKE, 256
    a.out, a.out_row, a.err = 3 * FAKE, 64, 4 * FAKE
    a.T, a.N, a.K, a.dtype, a.out_dtype = 5, 64, 256, L.MOE_BF16, L.MOE_BF16
    for n, v in kw.items():
        setattr(a, n, v)
    return L.lib().moe_linear(ctypes.byref(a), None)


E4M3 = dict(dtype=3, x_scale=5 * FAKE, w_scale=6 * FAKE)


@pytest.mark.parametrize("status,kw", [
    (ARG, dict(T=-1)), (ARG, dict(N=0)), (ARG, dict(K=0)), (ARG, dict(dtype=2)),
    (ARG, dict(dtype=4)), (ARG, dict(out_dtype=1)), (ARG, dict(out_dtype=3)),
    (ARG, dict(act=-1)), (ARG, dict(act=5)), (ARG, dict(x=None)), (ARG, dict(w=None)),
    (ARG, dict(out=None)), (ARG, dict(err=None)), (ARG, dict(x_scale=FAKE)),
    (ARG, dict(w_scale=FAKE)), (ARG, dict(E4M3, x_scale=None)), (ARG, dict(E4M3, w_scale=None)),
    (ARG, dict(out=FAKE)), (ARG, dict(out=2 * FAKE)),
    (ARG, dict(add=3 * FAKE, add_row=128)),                  # in place, another stride
    (SHAPE, dict(K=252)), (SHAPE, dict(E4M3, K=248)), (SHAPE, dict(K=65544, x_row=65544, w_row=65544)),
    (SHAPE, dict(T=(1 << 30) + 1)), (SHAPE, dict(N=(1 << 30) + 1, out_row=1 << 31)),
    (SHAPE, dict(x_row=248)), (SHAPE, dict(w_row=0)), (SHAPE, dict(out_row=63)),
    (SHAPE, dict(add=7 * FAKE, add_row=-64)), (SHAPE, dict(x_row=1 << 40)),
    (ALIGN, dict(x=FAKE + 8)), (ALIGN, dict(w=FAKE + 2)), (ALIGN, dict(x_row=260)),
    (ALIGN, dict(w_row=257)), (ALIGN, dict(out=3 * FAKE + 1)), (ALIGN, dict(bias=FAKE + 2)),
    (ALIGN, dict(add=7 * FAKE + 1, add_row=64)), (ALIGN, dict(E4M3, x_scale=FAKE + 1)),
    (ALIGN, dict(E4M3, x_row=264)), (ALIGN, dict(out_dtype=2, out=3 * FAKE + 2)),
])
def test_refusals(L, status, kw):
    assert _call(L, **kw) == status


def test_no_tokens_is_nothing(L):
    assert _call(L, T=0, x=None, out=None) == 0
    assert L.lib().moe_linear(None, None) == ARG


def test_binding_refuses_what_does_not_fit(L):
    w = torch.zeros((8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="Linear: weight must be"):
        L.Linear(None)
    with pytest.raises(ValueError, match="Linear: weight must be"):
        L.Linear(w.float())
    with pytest.raises(ValueError, match="CUDA"):
        L.Linear(w)
    assert ctypes.sizeof(L.LinearC) == L._LINEAR.size


@pytest.mark.parametrize("dtype,out", [(0, 0), (0, 2), (3, 0), (3, 2)])
def test_layouts_fit_the_multiprocessor(L, dtype, out):
    # shared memory within the limit and in proportion to tensor memory (blocks that run side
    # by side never wait for columns), accumulators within it, K split no finer than its chunks
    sizes = sorted({1, 2, 15, 16, 17, 33, 64, 100, 128, 250, 256, 257, 300, 512, 1000, 2047, 4096, 8191})
    for T in sizes + [70000, 1 << 24]:
        for N in (1, 127, 128, 129, 256, 2048, 2560, 8192, 16384, 100000):
            for K in (16, 64, 80, 128, 512, 2048, 8192, 65536):
                p = L.moe_debug_linear_plan(T, N, K, dtype, out)
                chunks = -(-K // (128 if dtype == 3 else 64))
                assert p["cols"] % 16 == 0 and 16 <= p["cols"] <= 256
                assert p["acc"] >= p["cols"] and p["acc"] & (p["acc"] - 1) == 0
                assert 32 <= p["tcols"] <= 512 and p["tcols"] & (p["tcols"] - 1) == 0
                assert p["tcols"] >= (p["acc"] if p["splits"] > 1 and out != 2 else 2 * p["acc"])
                assert p["splits"] in (1, 2, 4, 8) and p["splits"] <= chunks
                assert p["cols"] % p["splits"] == 0 and 2 <= p["stages"] <= 12
                assert (p["mode"] == 1) == (p["splits"] > 1)
                assert p["mode"] != 2 or p["cols"] % 32 == 0
                stage = (128 + p["cols"] // (2 if p["mode"] == 2 else 1)) * 128
                assert 1 <= p["sub"] <= 4 and p["smem"] >= p["stages"] * p["sub"] * stage + 1024
                if p["splits"] > 1:           # the partial sums fit into the ring
                    assert p["stages"] * p["sub"] * stage >= p["cols"] * 512
                assert p["smem"] <= 227 * 1024
                assert (p["smem"] + 1024) * 512 >= p["tcols"] * 228 * 1024
