"""Attention with sharp scores: bounds from the arithmetic that each kernel uses, tight enough
that a misplaced softmax reference, scale or rounding of a key shows."""
import pytest
import torch

from kv_case import Case

pytestmark = pytest.mark.gpu

FORMATS = [(64, 8), (64, 4), (128, 8), (128, 4), (256, 8), (256, 4)]


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("size,scale", [(30.0, None), (1.0, 2.0), (1.0, -0.7), (5.0, None)])
def test_few_rows(D, bits, size, scale):
    # Codes, scales, biases and queries enter the logits exactly; their sums are fp32, of
    # terms up to a few times |q| |k| (a code and its bias cancel in part): 2^-18 covers
    # 2^-24 of D + 10 roundings each at these D. Logits reach hundreds, so one wrong in its
    # 12th bit would move its weight by more than the bound.
    def shape(x, what, b):
        x[:, 0] *= size
    c = Case(D + bits, [700, 40, 3], 8, 2, D, bits, 16, prefix=300, nq=2, shape=shape)
    assert c.rows_kernel() == 0
    c.check(c.run(scale=scale), scale, keys=2.0 ** -18)


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("size", [2.0, 5.0])
def test_many_rows(D, bits, size):
    # Keys are rounded to fp16 (2^-11 of each element that is not far below its run's
    # largest). In the mean square a logit of size s errs by 2^-12.3 s, below 0.002 for
    # s = 5 nat, a weight by the same part of itself, and the outputs by less.
    def shape(x, what, b):
        x[:, 0] *= size
    c = Case(D + bits, [2500, 129, 700], 8, 2, D, bits, 16, nq=130, shape=shape)
    assert c.rows_kernel() == 2
    c.check(c.run(), keys=2.0 ** -10, norm=4e-3)
