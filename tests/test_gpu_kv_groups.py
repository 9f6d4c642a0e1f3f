"""Attention over values whose groups and tokens differ in size. Errors are taken per value
group: what a large group or token rounds must not show in a small one."""
import pytest
import torch

from kv_case import Case

pytestmark = pytest.mark.gpu

FORMATS = [(64, 8), (64, 4), (128, 8), (128, 4), (256, 8), (256, 4)]
# lens, query tokens, query heads per key/value head, prefix
FEW = {
    "one_token": ([700, 33, 1], 1, 8, 0),
    "drafts": ([400, 5, 90], 4, 4, 0),
    "prefix": ([90, 0, 17, 200], 1, 6, 500),
}
# the kernel for many query rows: its own tokens, its own and a prefix, a prefix alone
MANY = {
    "chunk": ([2600, 0, 1100], 130, 4, 0, 2),
    "chunk_and_prefix": ([2500, 39, 1300], 40, 8, 3000, 3),
    "prefix": ([(37 * b) % 300 for b in range(40)], 1, 8, 7000, 1),
}


def make_many(form, D, bits, **kw):
    lens, nq, G, prefix, where = MANY[form]
    return make((lens, nq, G, prefix), D, bits, where, **kw)


def make(form, D, bits, where=0, **kw):
    lens, nq, G, prefix = form
    c = Case(D + bits, lens, 2 * G, 2, D, bits, 32, prefix=prefix, nq=nq, **kw)
    assert c.rows_kernel() == where
    return c


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("form", list(FEW))
@pytest.mark.parametrize("power", [-24, -14, -8, 8, 20])
def test_groups_of_different_size(power, form, D, bits):
    def shape(x, what, b):
        x[:, 1, :, -64:] *= 2.0 ** power
    c = make(FEW[form], D, bits, shape=shape)
    c.check(c.run())


def outweighed(x, what, b, tokens, power):
    """`tokens` hold values 2^power larger, and logits far below the others' (query element 0
    is 8, so that a key element 0 of k adds 8 k / sqrt(D) to the logit)."""
    x[..., 0, :, 0] = 0.0
    at = tokens(x.shape[0])
    x[at, 1] *= 2.0 ** power
    x[at, 0, :, 0] = -5.0 * x.shape[-1] ** 0.5


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("tokens", ["first", "block", "spread"])
def test_large_values_that_are_outweighed(tokens, D, bits):
    # weights of e^-40 = 2^-57 times values of 2^20: nothing of them is left in the outputs
    at = {"first": lambda n: slice(0, 1), "block": lambda n: slice(0, min(40, n // 2)),
          "spread": lambda n: slice(0, n - 1, 37)}[tokens]
    c = make(FEW["one_token"], D, bits, shape=lambda x, w, b: outweighed(x, w, b, at, 20)
             if x.shape[0] > 1 else None)
    c.q[..., 0] = 8.0
    c.check(c.run())


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("form", list(FEW))
def test_one_group_large_in_some_tokens(form, D, bits):
    def shape(x, what, b):
        x[5::37, 1, :, :64] *= 2.0 ** 14
    c = make(FEW[form], D, bits, shape=shape)
    c.check(c.run(), norm=4e-3)


@pytest.mark.parametrize("D,bits", FORMATS)
def test_small_values_beside_zeros(D, bits):
    def shape(x, what, b):
        x[:, 1] *= 2.0 ** -14
        x[32:64, 1] = 0.0
        x[3::11, 1] = 0.0
    c = make(FEW["one_token"], D, bits, shape=shape)
    c.check(c.run())


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("what", ["scale", "bias"])
def test_rows_that_do_not_see_a_nan(what, D, bits):
    # the last of four query tokens alone sees the last token
    def words(scale, bias, where, b):
        if b == 0:
            (scale if what == "scale" else bias)[-1, 1, 0, 0] = torch.nan
    c = make(FEW["drafts"], D, bits, words=words)
    out = c.run()
    c.check(out)
    assert out[3].isnan().any() and not out[:3].isnan().any()


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("form", list(MANY))
@pytest.mark.parametrize("power", [-24, -14, -8, 8, 20])
def test_many_rows_groups_of_different_size(power, form, D, bits):
    def shape(x, what, b):
        x[:, 1, :, -64:] *= 2.0 ** power
    c = make_many(form, D, bits, shape=shape)
    c.check(c.run())


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("tokens", ["first", "block", "spread"])
def test_many_rows_large_values_that_are_outweighed(tokens, D, bits):
    # (tiles that hold both sizes multiply with bf16 weights and values)
    at = {"first": lambda n: slice(0, 1), "block": lambda n: slice(0, min(300, n // 2)),
          "spread": lambda n: slice(0, n - 1, 37)}[tokens]
    c = make_many("chunk", D, bits, shape=lambda x, w, b: outweighed(x, w, b, at, 20)
                  if x.shape[0] > 1 else None)
    c.q[..., 0] = 8.0
    c.check(c.run(), norm=4e-3, weights=2.0 ** -6)


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("form", list(MANY))
def test_many_rows_one_group_large_in_some_tokens(form, D, bits):
    def shape(x, what, b):
        x[5::137, 1, :, :64] *= 2.0 ** 14
    c = make_many(form, D, bits, shape=shape)
    c.check(c.run(), norm=4e-3, weights=2.0 ** -6)


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("form", list(MANY))
def test_many_rows_small_values_beside_zeros(form, D, bits):
    def shape(x, what, b):
        x[:, 1] *= 2.0 ** -14
        x[32:64, 1] = 0.0
        x[300:333, 1] = 0.0
        x[3::11, 1] = 0.0
    c = make_many(form, D, bits, shape=shape)
    c.check(c.run())


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("drift", [-1.0, 1.0])
def test_many_rows_values_that_drift(drift, D, bits):
    # sizes that leave any window around the first tile's
    def shape(x, what, b):
        t = torch.arange(x.shape[0], device="cuda", dtype=torch.float64)
        x[:, 1] *= torch.exp2(drift * t / 64)[:, None, None]
    c = make_many("chunk", D, bits, shape=shape)
    c.check(c.run(), norm=4e-3, weights=2.0 ** -6)


@pytest.mark.parametrize("D,bits", FORMATS)
def test_drafts_values_that_drift(D, bits):
    def shape(x, what, b):
        t = torch.arange(x.shape[0], device="cuda", dtype=torch.float64)
        x[:, 1] *= torch.exp2((1 - 2 * (b & 1)) * t / 16)[:, None, None]
    c = make(FEW["drafts"], D, bits, shape=shape)
    c.check(c.run())
