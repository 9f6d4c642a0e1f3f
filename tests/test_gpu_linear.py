"""moe_linear against float64.

Sizes and layouts are checked with small whole numbers, whose sums fp32 holds exactly: the
result is the rounded exact one, bit for bit. Other values: the accumulator adds 32 bytes of K
(16 or 32 products) at a time, so its sum is off by at most the number of those steps, plus a
tree of 6 within one and 8 for a split, times 2^-23 (it may truncate) of the sum of the
products' magnitudes. Activations change by at most 1.13 times their argument's error, and
their own arithmetic adds at most 2^-20 of the argument; one rounding of eps / 2 follows.
"""
import math

import pytest
import torch

from routing_q4_grouped_gb300 import moeq4

pytestmark = pytest.mark.gpu

ACTS = [moeq4.MOE_ACT_NONE, moeq4.MOE_ACT_RELU, moeq4.MOE_ACT_SILU, moeq4.MOE_ACT_GELU,
        moeq4.MOE_ACT_GELU_TANH]
BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def _whole(shape, top, g, dt):
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").float().to(dt)


def _case(T, N, K, dt, gap=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + 11 * N + 13 * K)
    x = _whole((T, K + gap), 3, g, dt)[:, :K]
    w = _whole((N, K + gap), 2, g, dt)[:, :K]
    return x, w, g


def _scales(T, N, dt, g):
    """Powers of two: exact products."""
    if dt is not E4M3:
        return None, None
    return (2.0 ** torch.randint(-3, 4, (T,), generator=g, device="cuda"),
            2.0 ** torch.randint(-3, 4, (N,), generator=g, device="cuda"))


def _exact(x, w, xs=None, ws=None):
    y = x.double() @ w.double().t()
    return y if xs is None else y * xs.double()[:, None] * ws.double()[None]


def _whole_check(T, N, K, dt, out_dt=F32, gap=0, bias=False, add=False):
    x, w, g = _case(T, N, K, dt, gap)
    xs, ws = _scales(T, N, dt, g)
    b = _whole((N,), 8, g, F32) if bias else None
    r = _whole((T, N), 8, g, out_dt) if add else None
    out = torch.full((T, N), 77.0, dtype=out_dt, device="cuda")
    lin = moeq4.Linear(w, b, ws)
    moeq4.moe_linear(x, lin, out, add=r, x_scale=xs)
    assert moeq4.moe_get_device_error(lin) == 0
    want = _exact(x, w, xs, ws)
    if bias:
        want = want + b.double()
    if add:
        want = want + r.double()
    assert torch.equal(out, want.to(F32).to(out_dt)), (out - want).abs().max()


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 63, 100, 129, 255, 257, 700])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 64), (127, 208), (128, 128), (129, 1040), (300, 512),
                                 (256, 2048)])
def test_sizes(T, N, K, dt):
    _whole_check(T, N, K, dt)


@pytest.mark.parametrize("T,N,K", [(1, 2560, 2048), (5, 2048, 8192), (64, 2048, 2048), (1, 16384, 512),
                                   (2047, 256, 2048), (1500, 2500, 1000), (4096, 512, 256),
                                   (3, 70000, 64), (33000, 130, 72)])
@pytest.mark.parametrize("dt,out_dt", [(BF16, BF16), (F16, F16), (F16, F32), (E4M3, BF16), (E4M3, F16)])
def test_large_sizes_and_types(T, N, K, dt, out_dt):
    if dt is E4M3:
        K = (K + 15) // 16 * 16
    _whole_check(T, N, K, dt, out_dt, bias=True, add=True)


@pytest.mark.parametrize("K", [8, 24, 56, 72, 120, 136])
def test_short_and_ragged_k(K):
    for T in (1, 40, 300):
        _whole_check(T, 200, K, BF16, gap=8)
        _whole_check(T, 200, K, F16, F16)


@pytest.mark.parametrize("T", [1, 50, 600])
def test_strides_and_rows_around(T):
    x, w, g = _case(T, 200, 512, BF16, gap=64)
    buf = torch.full((T + 2, 333), 5.0, dtype=BF16, device="cuda")
    out = buf[1:T + 1, 7:207]                     # odd alignment and stride
    add = _whole((1, 200), 4, g, BF16).expand(T, 200)
    moeq4.moe_linear(x, moeq4.Linear(w), out, add=add)
    assert torch.equal(out, (_exact(x, w) + add.double()).to(BF16))
    out.fill_(5.0)
    assert (buf == 5.0).all()


@pytest.mark.parametrize("T", [1, 64, 700])
def test_residual_in_place(T):
    x, w, g = _case(T, 256, 256, BF16)
    h = _whole((T, 256), 20, g, BF16)
    want = (_exact(x, w) + h.double()).to(BF16)
    moeq4.moe_linear(x, moeq4.Linear(w), h, add=h)
    assert torch.equal(h, want)


def _act64(y, act):
    if act == moeq4.MOE_ACT_RELU:
        return y.clamp(min=0)
    if act == moeq4.MOE_ACT_SILU:
        return y / (1 + (-y).exp())
    if act == moeq4.MOE_ACT_GELU:
        return 0.5 * y * torch.erfc(-y * math.sqrt(0.5))
    if act == moeq4.MOE_ACT_GELU_TANH:
        return 0.5 * y * (1 + (math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)).tanh())
    return y


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt,out_dt", [(BF16, BF16), (BF16, F32), (F16, F16), (E4M3, BF16), (E4M3, F32)])
def test_values(act, dt, out_dt):
    for T, N, K in ((1, 384, 2048), (77, 200, 400), (1300, 520, 1024)):
        g = torch.Generator(device="cuda").manual_seed(T)
        x = torch.randn((T, K), generator=g, device="cuda")
        w = torch.randn((N, K), generator=g, device="cuda") * K ** -0.5
        xs = ws = None
        if dt is E4M3:
            xs = torch.rand(T, generator=g, device="cuda") + 0.5
            ws = torch.rand(N, generator=g, device="cuda") * 0.02
            w = w * 50
        x, w = x.to(dt), w.to(dt)
        b = torch.randn(N, generator=g, device="cuda")
        r = torch.randn((T, N), generator=g, device="cuda").to(out_dt)
        out = torch.empty((T, N), dtype=out_dt, device="cuda")
        moeq4.moe_linear(x, moeq4.Linear(w, b, ws), out, act, r, xs)
        y = _exact(x, w, xs, ws) + b.double()
        size = _exact(x.double().abs(), w.double().abs(), xs, ws)
        steps = -(-K // (32 if dt is E4M3 else 16)) + 14
        arg = size * steps * 2.0 ** -23 + y.abs() * 2.0 ** -22 + b.double().abs() * 2.0 ** -24
        want = _act64(y, act) + r.double()
        bound = 1.13 * arg + y.abs() * 2.0 ** -20 + want.abs() * 2.0 ** -24
        bound = bound + (want.abs() + bound) * torch.finfo(out_dt).eps / 2 + 2.0 ** -25
        assert ((out.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("dt", [BF16, E4M3])
def test_accumulator_keeps_32_bits(dt):
    # 1 + 2^-k over a long K: an accumulator of fewer bits loses the small terms. The large
    # product comes first, so each of the others is added beside it.
    K = 4096
    x = torch.zeros((20, K), device="cuda")
    w = torch.zeros((40, K), device="cuda")
    x[:, 0] = w[:, 0] = 1.0
    x[:, 64:], w[:, 64:] = 2.0 ** -6, 2.0 ** -6       # e4m3 holds both
    out = torch.empty((20, 40), device="cuda")
    one = torch.ones
    lin = moeq4.Linear(w.to(dt), None, one(40, device="cuda") if dt is E4M3 else None)
    moeq4.moe_linear(x.to(dt), lin, out, x_scale=one(20, device="cuda") if dt is E4M3 else None)
    want = 1 + (K - 64) * 2.0 ** -12
    # each step of at most 32 products adds one error of 2^-23 of the sum
    assert (out - want).abs().max() <= want * (K // 16 + 8) * 2.0 ** -23


@pytest.mark.parametrize("T", [3, 40, 400])
def test_infinities_and_nans_stay_in_their_row(T):
    x, w, _ = _case(T, 130, 320, BF16)
    clean = _exact(x, w).to(BF16)
    x[1, 5], x[2, 300] = math.inf, math.nan
    for act in ACTS:
        out = torch.empty((T, 130), dtype=BF16, device="cuda")
        lin = moeq4.Linear(w)
        moeq4.moe_linear(x, lin, out, act)
        assert out[2].isnan().all() and not out[1].isfinite()[w[:, 5].float() > 0].any()
        if act == moeq4.MOE_ACT_NONE:
            rest = [i for i in range(T) if i not in (1, 2)]
            assert torch.equal(out[rest], clean[rest])
        assert moeq4.moe_get_device_error(lin) == 0


def test_activations_at_the_ends():
    # a product of one: the argument itself, from far below to far above
    x = torch.tensor([-3e38, -200.0, -20.0, -6.0, 0.0, 6.0, 20.0, 200.0, 3e38], device="cuda")
    X = torch.zeros((9, 8), dtype=BF16, device="cuda")
    X[:, 0] = x
    w = torch.zeros((1, 8), dtype=BF16, device="cuda")
    w[0, 0] = 1.0
    for act in ACTS:
        out = torch.empty((9, 1), device="cuda")
        moeq4.moe_linear(X, moeq4.Linear(w), out, act)
        y = X[:, 0].double()
        want = torch.where(y < -100, torch.zeros_like(y), _act64(y.clamp(-1e100, 1e100), act)) \
            if act else y
        want = torch.where((y > 100) & (act != 0), y, want)
        assert ((out[:, 0].double() - want).abs() <= y.abs().clamp(max=30) * 2.0 ** -20 +
                want.abs() * 2.0 ** -23).all(), (act, out[:, 0], want)


def test_no_tokens():
    w = torch.zeros((8, 64), dtype=BF16, device="cuda")
    e = torch.empty((0, 64), dtype=BF16, device="cuda")
    moeq4.moe_linear(e, moeq4.Linear(w), torch.empty((0, 8), dtype=BF16, device="cuda"))


def test_streams_side_by_side():
    # calls that split K over clusters, on two streams at once, many times
    x, w, _ = _case(17, 2048, 2048, BF16)
    x2, w2, _ = _case(90, 1000, 4096, BF16)
    a, b = (torch.empty((17, 2048), device="cuda") for _ in range(2))
    c, d = (torch.empty((90, 1000), device="cuda") for _ in range(2))
    l1, l2 = moeq4.Linear(w), moeq4.Linear(w2)
    moeq4.moe_linear(x, l1, a)
    moeq4.moe_linear(x2, l2, c)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(50):
        moeq4.moe_linear(x, l1, b, stream=s1)
        moeq4.moe_linear(x2, l2, d, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(c, d)
    assert moeq4.moe_get_device_error(l1) == 0 and moeq4.moe_get_device_error(l2) == 0


def test_captured():
    x, w, _ = _case(33, 640, 1024, BF16)
    out, want = (torch.empty((33, 640), dtype=BF16, device="cuda") for _ in range(2))
    lin = moeq4.Linear(w)
    moeq4.moe_linear(x, lin, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moeq4.moe_linear(x, lin, out)
        moeq4.moe_linear(x, lin, out, add=out)
    for i in range(3):
        x.mul_(-1 if i else 1)
        g.replay()
        moeq4.moe_linear(x, lin, want)
        moeq4.moe_linear(x, lin, want, add=want)
        assert torch.equal(out, want)


def test_binding_refusals():
    x, w, _ = _case(4, 64, 128, BF16)
    lin = moeq4.Linear(w)
    out = torch.empty((4, 64), dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="x must be"):
        moeq4.moe_linear(x[:, :64], lin, out)
    with pytest.raises(ValueError, match="out must be"):
        moeq4.moe_linear(x, lin, out[:, :63])
    with pytest.raises(ValueError, match="add must be"):
        moeq4.moe_linear(x, lin, out, add=out.float())
    with pytest.raises(ValueError, match="x_scale goes"):
        moeq4.moe_linear(x, lin, out, x_scale=torch.ones(4, device="cuda"))
    with pytest.raises(moeq4.MoeError):
        moeq4.moe_linear(x, lin, torch.empty((4, 64), dtype=F16, device="cuda"))
    with pytest.raises(ValueError, match="scale goes"):
        moeq4.Linear(w.to(E4M3))
    with pytest.raises(ValueError, match="bias must hold"):
        moeq4.Linear(w, torch.zeros(63, device="cuda"))


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("T,N,K", [(1, 256, 2048), (12, 128, 8192), (64, 512, 4096), (300, 256, 2048),
                                   (2047, 256, 4096), (3000, 2048, 1024), (700, 384, 16384)])
def test_fp32_results_of_long_sums(T, N, K, dt):
    # sums whose terms have one sign: what each step cuts off adds up. A piece has 32 steps, each
    # of which cuts off at most 2^-23 of the sum so far; the pieces' additions, at most 64 of them,
    # round by 2^-24 of theirs: 32 / 2 * 2^-23 (a sum that grows) + 64 / 2 * 2^-24 = 2^-18, and the
    # products within one step are added with a few more (4 of 2^-23).
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.rand((T, K), generator=g, device="cuda").to(dt)
    w = torch.rand((N, K), generator=g, device="cuda").to(dt)
    one = torch.ones(max(T, N), device="cuda")
    lin = moeq4.Linear(w, None, one[:N].clone() if dt is E4M3 else None)
    out = torch.empty((T, N), device="cuda")
    moeq4.moe_linear(x, lin, out, x_scale=one[:T].clone() if dt is E4M3 else None)
    want = _exact(x, w)
    assert ((out.double() - want).abs() <= want * (2.0 ** -18 + 2.0 ** -21)).all()


@pytest.mark.parametrize("T,step", [(3, 1 << 31), (40, (1 << 27) + 64), (300, (1 << 24) + 8)])
def test_far_rows(T, step):
    # element offsets past 2^31 in x, the residual and the result
    N, K = 200, 128
    big = torch.empty(step * (T - 1) + 1024, dtype=BF16, device="cuda")
    x, out = big.as_strided((T, K), (step, 1)), big.as_strided((T, N), (step, 1), 512)
    add = big.as_strided((T, N), (step, 1), 768)
    x0, w, g = _case(T, N, K, BF16)
    x.copy_(x0)
    add.copy_(_whole((T, N), 8, g, BF16))
    want = (_exact(x0, w) + add.double()).to(BF16)
    moeq4.moe_linear(x, moeq4.Linear(w), out, add=add)
    assert torch.equal(out, want) and torch.equal(x, x0)


def test_far_weights():
    # weight rows 2^31 elements and more away from the first
    N, K, step = 130, 256, (1 << 24) + 8
    big = torch.empty(step * (N - 1) + K, dtype=BF16, device="cuda")
    w = big.as_strided((N, K), (step, 1))
    for T in (2, 60):
        x, w0, _ = _case(T, N, K, BF16)
        w.copy_(w0)
        out = torch.empty((T, N), device="cuda")
        moeq4.moe_linear(x, moeq4.Linear(w), out)
        assert torch.equal(out, _exact(x, w0).float())
