"""moe_rms_norm against the formula in float64.

Tolerances, relative to the value. An fp32 sum of up to 16384 squares is taken as at most
32 terms per thread and a tree of at most 5 + 16 additions, so the root of its mean is off by
at most (32 + 21) / 2 roundings; the root, two products and the weight's sum add 5: below
32 * 2^-24 = 2^-19. Then one rounding to the type (eps / 2 of the value, or half the smallest
step), or to e4m3 (2^-4 of the value, or half of 2^-9 scales).
"""
import math

import pytest
import torch

from routing_q4_grouped_gb300 import moeq4

pytestmark = pytest.mark.gpu

ARITH = 2.0 ** -19
STEP = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def _ref(x, add, weight, eps, offset):
    h = x.double() if add is None else x.double() + add.double()
    gain = (1.0 if weight is None else weight.double()) + offset
    return h, h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * gain


def _near(got, want, more=0.0):
    dt = got.dtype
    bound = want.abs() * (torch.finfo(dt).eps / 2 * (1 + ARITH) + more) + STEP[dt]
    bad = (got.double() - want).abs() > bound
    assert not bad.any(), (got[bad][:4], want[bad][:4], int(bad.sum()))


def _check_codes(codes, scales, y):
    s = scales.double()
    top = y.abs().amax(-1)
    want = (top / 448.0).clamp(min=2.0 ** -126)
    assert ((s - want).abs() <= want * 2 * ARITH).all()
    got = codes.double() * s[..., None]
    bound = (y.abs() * 2.0 ** -4).maximum(s[..., None] * 2.0 ** -10) * (1 + 4 * ARITH)
    # the largest element may be pushed over 448 scales by the arithmetic and is then 448
    assert ((got - y).abs() <= bound + 2 * ARITH * y.abs()).all()


def _inputs(T, H, D, dt, add, weight, gap=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T * 131 + D)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")      # noqa: E731
    x = rnd(T, H + gap, D).to(dt)[:, :H]
    return (x, rnd(T, H, D).to(dt) if add else None,
            (1 + 0.2 * rnd(D)).to(dt) if weight else None)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,D,gap", [
    (1, 1, 1, 0), (3, 1, 7, 0), (1, 1, 2048, 0), (5, 1, 64, 0), (9, 3, 128, 1), (7, 2, 96, 0),
    (17, 5, 256, 2), (4, 1, 511, 0), (2, 1, 512, 0), (3, 1, 1024, 0), (3, 1, 1032, 0),
    (2, 1, 4095, 0), (2, 1, 4097, 1), (2, 1, 5120, 0), (2, 1, 8192, 0), (2, 1, 8200, 0),
    (1, 1, 16383, 0), (2, 1, 16384, 0), (513, 4, 80, 1)])
def test_shapes(T, H, D, gap, dt):
    x, add, weight = _inputs(T, H, D, dt, True, True, gap)
    out, total = torch.empty_like(add), torch.empty_like(add)
    codes = torch.empty(add.shape, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((T, H), device="cuda")
    moeq4.moe_rms_norm(x, weight, out, add, total, codes, scales, eps=1e-5, offset=0.25)
    h, y = _ref(x, add, weight, 1e-5, 0.25)
    _near(total, h, 2.0 ** -24)
    _near(out, y, ARITH)
    _check_codes(codes, scales, y)


@pytest.mark.parametrize("add,weight,offset", [(False, False, 0.0), (False, True, 1.0),
                                               (True, False, -0.5)])
def test_parts_left_out(add, weight, offset):
    x, a, w = _inputs(33, 2, 192, torch.bfloat16, add, weight)
    out = torch.full_like(x, 7.0)
    moeq4.moe_rms_norm(x, w, out, a, offset=offset)
    _near(out, _ref(x, a, w, 1e-6, offset)[1], ARITH)
    # the same bits without any other result, and codes alone
    codes = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((33, 2), device="cuda")
    moeq4.moe_rms_norm(x, w, add=a, codes=codes, scales=scales, offset=offset)
    _check_codes(codes, scales, _ref(x, a, w, 1e-6, offset)[1])


@pytest.mark.parametrize("D", [128, 2048, 2047])
def test_in_place_and_two_dimensions(D):
    x, add, weight = _inputs(65, 1, D, torch.bfloat16, True, True)
    x, add = x[:, 0], add[:, 0]
    out, total = torch.empty_like(add), torch.empty_like(add)
    moeq4.moe_rms_norm(x, weight, out, add, total)
    x2, add2 = x.clone(), add.clone()
    moeq4.moe_rms_norm(x2, weight, x2, add2, add2)      # the norm over x, the sum over add
    assert torch.equal(x2, out) and torch.equal(add2, total)
    x3, add3 = x.clone(), add.clone()
    moeq4.moe_rms_norm(x3, weight, add3, add3, x3)
    assert torch.equal(add3, out) and torch.equal(x3, total)
    both = x.clone()
    moeq4.moe_rms_norm(both, weight, out, both)         # x + x
    _near(out, _ref(x, x, weight, 1e-6, 0.0)[1], ARITH)


def test_rows_around_are_left_alone():
    buf = torch.full((12, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    x = torch.randn((10, 5, 128), device="cuda").bfloat16()
    moeq4.moe_rms_norm(x, out=buf[1:11, 2:7])
    _near(buf[1:11, 2:7], _ref(x, None, None, 1e-6, 0.0)[1], ARITH)
    buf[1:11, 2:7] = 3.0
    assert (buf == 3.0).all()


def test_heads_outside_tokens():
    # heads as the outer axis: head stride above the row stride
    x = torch.randn((6, 40, 128), device="cuda").bfloat16().transpose(0, 1)
    out = torch.empty((6, 40, 128), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    moeq4.moe_rms_norm(x, out=out)
    _near(out, _ref(x, None, None, 1e-6, 0.0)[1], ARITH)


def test_broadcast_summand():
    x = torch.randn((9, 256), device="cuda").bfloat16()
    add = torch.randn((1, 256), device="cuda").bfloat16().expand(9, 256)
    out = torch.empty_like(x)
    moeq4.moe_rms_norm(x, out=out, add=add)
    _near(out, _ref(x, add, None, 1e-6, 0.0)[1], ARITH)


@pytest.mark.parametrize("D", [64, 4096])
@pytest.mark.parametrize("size", [1e-38, 1e-25, 1e-15, 1e15, 1e30, 1e37])
def test_squares_out_of_range(D, size):
    # squares below or above fp32's range; a row of ordinary size beside them
    x, _, _ = _inputs(6, 1, D, torch.float32, False, False)
    x = x * torch.tensor([1.0, size, size, 1.0, size, 1.0], device="cuda")[:, None, None]
    for eps in (1e-6, 1e-38):
        out = torch.empty_like(x)
        moeq4.moe_rms_norm(x, out=out, eps=eps)
        e32 = float(torch.tensor(eps, dtype=torch.float32))
        _near(out, _ref(x, None, None, e32, 0.0)[1], ARITH)


@pytest.mark.parametrize("D", [96, 2048])
def test_zeros_infinities_and_nans(D):
    x, _, _ = _inputs(6, 1, D, torch.bfloat16, False, False)
    x = x[:, 0].contiguous()
    x[1] = 0
    x[2, 5] = math.nan
    x[3, 7] = math.inf
    x[4, D - 1] = -math.inf
    out = torch.empty_like(x)
    codes = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(6, device="cuda")
    moeq4.moe_rms_norm(x, out=out, codes=codes, scales=scales)
    ok = [0, 1, 5]
    _near(out[ok], _ref(x[ok], None, None, 1e-6, 0.0)[1], ARITH)
    _check_codes(codes[ok], scales[ok], _ref(x[ok], None, None, 1e-6, 0.0)[1])
    assert (out[1] == 0).all() and scales[1] == 2.0 ** -126
    assert out[2].isnan().all()
    for r, c in ((3, 7), (4, D - 1)):
        assert out[r, c].isnan() and (out[r].float().nan_to_num() == 0).all()
    assert scales[2:5].isnan().all()


def test_no_tokens_and_far_rows():
    e = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    moeq4.moe_rms_norm(e, out=e)
    # element offsets past 2^31: two rows 2^31 elements apart
    big = torch.empty((1 << 31) + 256, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, 256), (1 << 31, 1))
    x.copy_(torch.randn((2, 256), device="cuda"))
    out = torch.empty((2, 256), dtype=torch.bfloat16, device="cuda")
    moeq4.moe_rms_norm(x, out=out)
    _near(out, _ref(x, None, None, 1e-6, 0.0)[1], ARITH)


def test_stream_and_graph():
    x, add, weight = _inputs(200, 1, 2048, torch.bfloat16, True, True)
    want, out = torch.empty_like(add), torch.empty_like(add)
    moeq4.moe_rms_norm(x, weight, want, add)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moeq4.moe_rms_norm(x, weight, out, add, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        moeq4.moe_rms_norm(x, weight, out, add)
    for _ in range(2):
        x.mul_(-1)
        add.mul_(-1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, -want) or torch.equal(out, want)
    assert torch.equal(out, want)


def test_binding_refusals():
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="out must be"):
        moeq4.moe_rms_norm(x, out=x.float())
    with pytest.raises(ValueError, match="weight must hold"):
        moeq4.moe_rms_norm(x, x[0, :64].contiguous(), x)
    with pytest.raises(ValueError, match="dense"):
        moeq4.moe_rms_norm(x[:, ::2], out=x[:, :64])
    with pytest.raises(ValueError, match="scales must be"):
        moeq4.moe_rms_norm(x, codes=x.to(torch.float8_e4m3fn), scales=torch.empty(3, device="cuda"))
    with pytest.raises(moeq4.MoeError):
        moeq4.moe_rms_norm(x)


@pytest.mark.parametrize("dt,T,H,D", [(torch.bfloat16, 9001, 1, 2048), (torch.float16, 3001, 3, 1200),
                                      (torch.float32, 7001, 1, 1024), (torch.bfloat16, 4100, 1, 8192)])
def test_many_long_rows(dt, T, H, D):
    # rows that a block goes through in turns; a row alone gives the same bits
    x, add, weight = _inputs(T, H, D, dt, True, True, gap=1)
    out, total = torch.empty_like(add), torch.empty_like(add)
    codes = torch.empty(add.shape, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((T, H), device="cuda")
    moeq4.moe_rms_norm(x, weight, out, add, total, codes, scales, eps=1e-5)
    some = torch.tensor([0, 1, T // 2, T - 2, T - 1])
    h, y = _ref(x[some], add[some], weight, 1e-5, 0.0)
    _near(total[some], h, 2.0 ** -24)
    _near(out[some], y, ARITH)
    _check_codes(codes[some], scales[some], y)
    for lo in range(0, T, 600):
        part = slice(lo, min(T, lo + 600))
        o, s2 = torch.empty_like(add[part]), torch.empty_like(add[part])
        c, sc = torch.empty_like(codes[part]), torch.empty_like(scales[part])
        moeq4.moe_rms_norm(x[part], weight, o, add[part], s2, c, sc, eps=1e-5)
        assert torch.equal(o, out[part]) and torch.equal(s2, total[part])
        assert torch.equal(c.view(torch.uint8), codes[part].view(torch.uint8))
        assert torch.equal(sc, scales[part])
    # in place: the norm over x's copy, the sum over add
    x2 = x.contiguous()
    moeq4.moe_rms_norm(x2, weight, x2, add, add, eps=1e-5)
    assert torch.equal(x2, out) and torch.equal(add, total)


def test_many_long_rows_without_summand():
    x, _, _ = _inputs(6000, 1, 4096, torch.bfloat16, False, False)
    x[5] = 0
    x[4000, 0, 7] = math.nan
    out = torch.empty_like(x)
    moeq4.moe_rms_norm(x, out=out)
    ok = [i for i in range(0, 6000, 37) if i != 4000]
    _near(out[ok], _ref(x[ok], None, None, 1e-6, 0.0)[1], ARITH)
    assert out[4000].isnan().all() and (out[5] == 0).all()


@pytest.mark.parametrize("D", [128, 130, 2048])
def test_codes_inside_wider_rows(D):
    # codes and results of heads inside rows of more heads; what lies between stays
    x, add, weight = _inputs(50, 3, D, torch.bfloat16, True, True, gap=1)
    rows = torch.full((50, 5, D), 2.0, device="cuda").to(torch.float8_e4m3fn)
    out = torch.full((50, 5, D), 2.0, dtype=torch.bfloat16, device="cuda")
    scales = torch.empty((50, 3), device="cuda")
    moeq4.moe_rms_norm(x, weight, out[:, 1:4], add, codes=rows[:, 1:4], scales=scales)
    y = _ref(x, add, weight, 1e-6, 0.0)[1]
    _near(out[:, 1:4], y, ARITH)
    _check_codes(rows[:, 1:4], scales, y)
    for t in (rows.float(), out.float()):
        assert (t[:, 0] == 2.0).all() and (t[:, 4] == 2.0).all()
