"""Attention by the kernel for many query rows: every head size and code width, units of one
and two query tiles, contexts in one piece and cut, a prefix beside own tokens, and the
tiles that need more than the plain path (NaN groups, missing pages, wide spreads)."""
import pytest
import torch

from kv_case import Case
from routing_q4_grouped_gb300 import moeq4

pytestmark = pytest.mark.gpu

FORMATS = [(64, 8), (64, 4), (128, 8), (128, 4), (256, 8), (256, 4)]

# lens, nq, query heads per key/value head, key/value heads, prefix, contexts on this kernel
FORMS = {
    "one_query_tile": ([22000], 12, 8, 2, 0, 2),
    "two_query_tiles": ([9000], 30, 8, 2, 0, 2),
    "mixed_tiles": ([3000, 0, 129, 700, 1], 130, 4, 2, 0, 2),
    "whole_units": ([600 - 7 * b for b in range(80)], 8, 8, 2, 0, 2),
    "shared_heads_odd": ([2111, 2500, 64], 27, 5, 5, 0, 2),
    "prefix_here_own_there": ([(37 * b) % 300 for b in range(40)], 1, 8, 2, 7000, 1),
    "prefix_and_own_here": ([2500, 39, 1300], 40, 8, 2, 3000, 3),
    "prefix_there_own_here": ([2500, 0, 1300], 40, 8, 2, 41, 2),
}


def make(form, D, bits, P=48, **kw):
    lens, nq, G, Hkv, prefix, where = FORMS[form]
    c = Case(D + bits + len(form), lens, G * Hkv, Hkv, D, bits, P, prefix=prefix, nq=nq, **kw)
    assert c.rows_kernel() == where
    return c


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("form", list(FORMS))
def test_forms(form, D, bits):
    c = make(form, D, bits)
    out = c.run()
    c.check(out)
    assert torch.equal(c.run().view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("P", [16, 32, 80, 256, 4096])
def test_page_sizes(P):
    make("mixed_tiles", 128, 8, P).check(make("mixed_tiles", 128, 8, P).run())


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("form", ["one_query_tile", "mixed_tiles", "prefix_here_own_there"])
def test_nan_values_and_keys(form, D, bits):
    # a NaN group reaches its own elements of the rows that see its token, a NaN key whole rows
    lens = FORMS[form][0]

    def words(scale, bias, what, b):
        n = scale.shape[0]
        if what == "prefix" and n:
            scale[n // 2, 1, 0, -1] = 0.0
            bias[n // 2, 1, 0, -1] = torch.nan
        if what == "own" and n > 1 and b in (0, 3):
            bias[n - 2, 1, 1, 0] = torch.nan                 # near the end: few rows see it
            bias[n - 1, 0, 0, 0] = torch.nan
    c = make(form, D, bits, words=words)
    out = c.run()
    c.check(out, norm=4e-3, weights=2.0 ** -6)
    assert out.isnan().any() and not out.isnan().all(), lens


@pytest.mark.parametrize("D,bits", FORMATS)
@pytest.mark.parametrize("form", ["two_query_tiles", "mixed_tiles", "prefix_here_own_there"])
def test_tokens_of_very_different_size(form, D, bits):
    def shape(x, what, b):
        n = x.shape[0]
        e = torch.arange(n, device="cuda")
        x[:, 0] *= torch.exp2(((e * 7) % 5 - 3.0))[:, None, None]          # keys 2^-3 .. 2
        x[:, 1] *= torch.exp2(((e * 5) % 19 - 9.0))[:, None, None]         # values 2^-9 .. 2^9
    c = make(form, D, bits, shape=shape)
    c.check(c.run(), norm=4e-3, weights=2.0 ** -6)


@pytest.mark.parametrize("D,bits", FORMATS)
def test_missing_pages(D, bits):
    c = make("mixed_tiles", D, bits)
    clean = c.run()
    c.table[0, 5] = c.cache.pages                            # tokens 240 .. 287 of request 0
    c.table[3, 1] = -1                                       # tokens 48 .. 95 of request 3
    c.seen_own[0][240:288] = False
    c.seen_own[3][48:96] = False
    out = c.run()
    c.check(out, norm=4e-3, weights=2.0 ** -6, err=moeq4.MOE_DEVERR_BAD_PAGE)
    nq = c.nq
    assert torch.equal(out[nq:3 * nq], clean[nq:3 * nq]) and torch.equal(out[4 * nq:], clean[4 * nq:])


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 60])
@pytest.mark.parametrize("D,bits", [(64, 4), (128, 8), (256, 4)])
def test_values_far_from_one(D, bits, size):
    def shape(x, what, b):
        x *= size
    c = make("mixed_tiles", D, bits, shape=shape)
    s = D ** -0.5 / size
    c.check(c.run(scale=s), s)


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.4])
def test_scales(scale):
    c = make("mixed_tiles", 128, 8)
    c.check(c.run(scale=scale), scale)


def test_max_len_is_only_a_bound():
    c = make("mixed_tiles", 128, 4)
    c.table = torch.cat((c.table, torch.full((5, 2000), 0x7FFFFFFF, dtype=torch.int32, device="cuda")), 1)
    assert c.rows_kernel(90000) == 2
    c.check(c.run(max_len=90000))


def test_lengths_outside_are_clamped_and_reported():
    c = make("mixed_tiles", 64, 8)
    clean = c.run()
    c.lens[0], c.lens[1] = 3001, -5
    out = c.run()
    assert moeq4.moe_get_device_error(c.cache) == moeq4.MOE_DEVERR_BAD_LENGTH
    assert torch.equal(out, clean)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", ["whole_units", "prefix_and_own_here"])
def test_strides_streams_and_graphs(form, D):
    c = make(form, D, 8)
    want = c.run()
    T, Hq = c.q.shape[:2]
    wide = torch.full((T, Hq + 4, D), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + Hq] = c.q
    out = torch.full((Hq, T, D + 8), 2.0, dtype=torch.bfloat16, device="cuda")
    view = out.transpose(0, 1)[..., :D]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(q=wide[:, 2:2 + Hq], out=view)
    side.synchronize()
    assert torch.equal(view, want) and (out[..., D:] == 2).all()
    ws = moeq4.alloc_workspace(moeq4.moe_kv_attention_workspace_size(
        c.B, c.nq, c.Hq, c.Hkv, D, c.max_len, c.prefix))
    dense = torch.zeros_like(want)
    c.run(out=dense, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=dense, ws=ws)
    dense.zero_()
    g.replay()
    assert torch.equal(dense, want)
