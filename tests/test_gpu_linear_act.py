"""Activations of moe_linear over their whole range, relative to their value.

Products of zeros and a bias: the activation's argument is the bias, an fp32 number, exactly.
The value is taken in float64 from a form that does not cancel (erfc, a sigmoid).

Bounds, in units u = 2^-24 (half an ulp at most). Next to 16-bit results, of which one rounding
follows, and with the errors CUDA states for __expf (2 + 1.2 |x| ulp) and __fdividef (2 ulp):

  silu       the exponential 2 (2 + 1.2 |y|), sum 1, quotient 4, product 1
  gelu_tanh  the same at the sigmoid's argument w, and w itself: 6 roundings of |w|
  gelu       a polynomial to 2^-16, its own arithmetic 32, the exponential of -y^2 / 2 with an
             argument that is off by 2 roundings

For fp32 results the exponential is expf (2 ulp), quotients are rounded:

  silu       9 (exponential 4, in the sum and in the product; sum, quotient and product)
  gelu_tanh  10, and 6 roundings of |w| times the sigmoid's sensitivity, 1 - sigmoid(w)
  gelu       32 (t 8, polynomial 16, exponential 4, products), and a rounding of y^2 / 2 where the
             tail is the result

An exponential below 2^-126 has fewer bits: 2^-149 of it, times |y| < 120, is the least that can
be told apart (2^-142).
"""
import math

import pytest
import torch

from routing_q4_grouped_gb300 import moeq4

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
SILU, GELU, TANH = moeq4.MOE_ACT_SILU, moeq4.MOE_ACT_GELU, moeq4.MOE_ACT_GELU_TANH
U = 2.0 ** -24
STEP = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 0.0}


def _arguments():
    near = torch.linspace(-14.0, 14.0, 2801, device="cuda")
    far = torch.linspace(-110.0, 110.0, 1101, device="cuda")
    small = torch.tensor([s * 10.0 ** -e for e in range(1, 38) for s in (1, -1)], device="cuda")
    large = torch.tensor([s * 10.0 ** e for e in range(2, 38) for s in (1, -1)], device="cuda")
    return torch.cat((near, far, small, large))


def _value(y, act):
    """(value, sigmoid's argument) in float64."""
    if act == GELU:
        return 0.5 * y * torch.special.erfc(-y * math.sqrt(0.5)), y * y / 2
    w = y if act == SILU else 2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)
    e = torch.exp(-w.abs())
    return y * torch.where(w < 0, e, 1.0) / (1 + e), w


def _bound(y, act, want, w, out_dt):
    size = w.abs().clamp(max=200.0)            # (beyond that every value is 0 or y)
    if out_dt is F32:
        if act == SILU:
            rel = 9 * U
        elif act == TANH:
            rel = (10 + 6 * size * torch.sigmoid(-w)) * U
        else:
            rel = (32 + size) * U
    else:
        slow = 2 * (2 + 1.2 * size)
        rel = (slow + 6) * U if act == SILU else (slow + 6 + 6 * size) * U if act == TANH else \
            2.0 ** -16 + (32 + slow + 2 * size) * U
        rel = rel + torch.finfo(out_dt).eps / 2 * (1 + rel)
    return want.abs() * rel + 2.0 ** -142 + STEP[out_dt]


def _run(y, T, dt, out_dt, act):
    K = 64
    one = torch.ones(max(T, y.numel()), device="cuda")
    scale = one[:y.numel()].clone() if dt is E4M3 else None
    lin = moeq4.Linear(torch.zeros((y.numel(), K), device="cuda").to(dt), y, scale)
    x = torch.zeros((T, K), device="cuda").to(dt)
    out = torch.empty((T, y.numel()), dtype=out_dt, device="cuda")
    moeq4.moe_linear(x, lin, out, act, x_scale=one[:T].clone() if dt is E4M3 else None)
    assert moeq4.moe_get_device_error(lin) == 0
    return out


@pytest.mark.parametrize("act", [SILU, GELU, TANH])
@pytest.mark.parametrize("dt,out_dt", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (E4M3, BF16),
                                       (E4M3, F16), (E4M3, F32)])
@pytest.mark.parametrize("T", [1, 12, 40, 300, 3000])
def test_relative_to_the_value(T, dt, out_dt, act):
    y = _arguments()
    if out_dt is F16:
        y = y[y.abs() < 6e4].contiguous()
    out = _run(y, T, dt, out_dt, act)
    assert torch.equal(out, out[:1].expand_as(out))
    want, w = _value(y.double(), act)
    off = (out[0].double() - want).abs()
    bad = off > _bound(y.double(), act, want, w, out_dt)
    assert not bad.any(), (y[bad][:5], out[0][bad][:5], want[bad][:5], int(bad.sum()))


@pytest.mark.parametrize("act", [SILU, GELU, TANH])
@pytest.mark.parametrize("out_dt", [BF16, F32])
def test_ends(act, out_dt):
    # +inf stays, -inf is 0 times infinity, NaN stays, zeros keep their sign
    y = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0], device="cuda")
    for T in (2, 200):
        out = _run(y, T, BF16, out_dt, act)[T - 1].float()
        assert out[0] == math.inf and out[1].isnan() and out[2].isnan()
        assert out[3] == 0 and out[4] == 0
