"""Rotary positions, the quantised cache and attention over it on the GPU, against
the float64 oracle. Error bounds are derived from the roundings of each step and
stand beside them."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from oracle import kv
from routing_q4_grouped_gb300 import moeq4

pytestmark = pytest.mark.gpu

# unit roundoff of each type: 2^-p with p significant bits (8, 11, 24)
DTYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "f16": (torch.float16, 2.0 ** -11),
          "f32": (torch.float32, 2.0 ** -24)}


def f64(t):
    return t.detach().double().cpu().numpy()


def bf16_tensor(a):
    return torch.from_numpy(np.asarray(a, np.float32)).cuda().bfloat16()


def rope_spec(rot, interleaved=False, base=1e4, mscale=1.0, **kw):
    ph = moeq4.moe_rope_phases(rot, base, **kw)
    return moeq4.RopeSpec(ph.cuda(), rot, interleaved, mscale), ph.numpy().view(np.uint64)


def rope_bound(x, y, rot, interleaved, mscale, unit):
    """Angle: float of a 32-bit fraction, one constant and one product, 3 roundings of
    at most pi * 2^-24 each; cos and sin to 2 ulp; mscale, product and sum roundings
    2^-24 each: below 1.2e-6 of (|a| + |b|) * mscale. Then the rounding of the type
    (unit relative, 2^-25 absolute for fp16's smallest numbers)."""
    a, b = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
            else (slice(0, rot // 2), slice(rot // 2, rot)))
    e = np.zeros(x.shape)
    e[..., a] = e[..., b] = 1.2e-6 * mscale * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return e + unit * (np.abs(y) + e) + 2.0 ** -25 * (unit > 1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 64, 64), (5, 3, 128, 64), (33, 2, 256, 136),
                                       (7, 5, 80, 6), (3, 2, 64, 2), (300, 18, 128, 128)])
def test_rope(dtype, interleaved, T, H, D, rot):
    dt, ulp = DTYPES[dtype]
    rng = np.random.default_rng(T * D + rot)
    qkv = torch.from_numpy(rng.standard_normal((T, H + 2, D)).astype(np.float32)).cuda().to(dt)
    x = qkv[:, 1:1 + H]
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    pos[0] = 0 if T > 1 else 2 ** 31 - 1
    spec, ph = rope_spec(rot, interleaved, mscale=1.25)
    for backward in (False, True):
        out = torch.full((T, H, D), 7.0, dtype=dt, device="cuda")
        moeq4.moe_rope(x, out, torch.from_numpy(pos).cuda(), spec, backward=backward)
        ref = kv.rope(f64(x), pos, ph, rot, interleaved, 1.25, backward)
        bound = rope_bound(f64(x), ref, rot, interleaved, 1.25, ulp)
        bound[..., rot:] = 0
        assert np.all(np.abs(f64(out) - ref) <= bound)
    # in place on a strided view: the same bits, and nothing beside it
    before = qkv.clone()
    moeq4.moe_rope(x, x, torch.from_numpy(pos).cuda(), spec, backward=True)
    assert torch.equal(x, out)
    assert torch.equal(qkv[:, 0], before[:, 0]) and torch.equal(qkv[:, 1 + H:], before[:, 1 + H:])


def test_rope_unaligned_rows_and_transposed_output():
    rng = np.random.default_rng(5)
    buf = torch.from_numpy(rng.standard_normal(4 * 3 * 131 + 1).astype(np.float32)).cuda().bfloat16()
    x = buf[1:].as_strided((4, 3, 128), (3 * 131, 131, 1), 1)
    out = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    pos = torch.tensor([0, 3, -5, 1 << 30], dtype=torch.int32, device="cuda")
    spec, ph = rope_spec(128)
    moeq4.moe_rope(x, out, pos, spec)
    ref = kv.rope(f64(x), pos.cpu().numpy(), ph, 128)
    assert np.all(np.abs(f64(out) - ref) <= rope_bound(f64(x), ref, 128, False, 1.0, 2.0 ** -8))


def test_rope_gradient_by_differences():
    # y is linear in x: (y(x + h e) - y(x - h e)) / 2h projected on g must equal R^T g
    # (fp32: differences of values near 1 with h = 0.5 lose 2^-23 each)
    rng = np.random.default_rng(6)
    spec, _ = rope_spec(16, True, mscale=1.1)
    x = torch.from_numpy(rng.standard_normal((1, 1, 64)).astype(np.float32)).cuda()
    g = torch.from_numpy(rng.standard_normal((1, 1, 64)).astype(np.float32)).cuda()
    pos = torch.tensor([12345], dtype=torch.int32, device="cuda")
    run = lambda a, back=False: [moeq4.moe_rope(a, o := torch.empty_like(a), pos, spec, back), o][1]
    grad = run(g, True)[0, 0]
    for e in range(20):
        d = torch.zeros_like(x)
        d[..., e] = 0.5
        num = float(((run(x + d).double() - run(x - d).double()) * g.double()).sum())
        assert abs(num - float(grad[e])) < 64 * 4 * 2.0 ** -23 * 4


def test_rope_of_nothing():
    spec, _ = rope_spec(64)
    x = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    moeq4.moe_rope(x, x, torch.empty(0, dtype=torch.int32, device="cuda"), spec)


# -------------------------------------------------------------------- cache

def quantised32(x, bits):
    """The write's own arithmetic in fp32 on given bf16 values: bit-exact values."""
    g = x.astype(np.float32).reshape(*x.shape[:-1], -1, 64)
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    levels = np.float32(2 ** bits - 1)
    half = np.float32(0.5)
    rng_ = hi * half - lo * half
    scale = O.bf16_value(O.to_bf16(rng_ * (np.float32(1) / (half * levels)))).astype(np.float32)
    with np.errstate(divide="ignore"):
        per = np.where(scale > 0, np.float32(1) / scale, np.float32(0))
    code = np.clip(np.rint((g - lo) * per), 0, levels)
    return (scale.astype(np.float64) * code + lo).reshape(x.shape)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,Hkv,Hq,P,T", [(64, 1, 1, 16, 1), (128, 2, 16, 16, 37), (256, 2, 6, 48, 100),
                                          (128, 8, 32, 64, 5), (64, 3, 3, 4096, 9)])
def test_append_then_read(bits, D, Hkv, Hq, P, T):
    rng = np.random.default_rng(D + T)
    qkv = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float32)).cuda().bfloat16()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pages = -(-T // P) + 2
    cache = moeq4.KVCache.alloc(pages, P, Hkv, D, bits)
    cache.data.fill_(255)
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    pos = rng.integers(0, 200000, T).astype(np.int32)
    if T > 4:
        slots[3] = -1
    st, pt = torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda()
    k_out, v_out = (torch.full((T, Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kept = slots >= 0

    # without positions: bit-exact against the same arithmetic on the host
    moeq4.moe_kv_append(cache, k, v, st)
    moeq4.moe_kv_read(cache, st, k_out, v_out)
    for x, got in ((k, k_out), (v, v_out)):
        want = O.bf16_value(O.to_bf16(quantised32(f64(x), bits)))
        want[~kept] = 0
        assert np.array_equal(f64(got), want)
    data = cache.data.cpu().numpy().reshape(pages, 2, Hkv, -1)
    rk, rv = kv.read_rows(data, slots[kept], P, D, bits)      # the documented layout
    assert np.array_equal(O.bf16_value(O.to_bf16(rk)), f64(k_out)[kept])
    assert np.array_equal(O.bf16_value(O.to_bf16(rv)), f64(v_out)[kept])
    # every byte that belongs to no written slot is as it was
    clean = np.full_like(data, 255)
    for s in slots[kept]:
        page, r = divmod(int(s), P)
        rb, nb = D * bits // 8, D // 64 * 4
        for at, n in ((r * rb, rb), (P * rb + r * nb, nb)):
            clean[page, :, :, at:at + n] = data[page, :, :, at:at + n]
    assert np.array_equal(clean, data)

    # with positions
    for inter in (False, True):
        for rot in {D, D // 2, D // 2 + 8}:
            spec, ph = rope_spec(rot, inter, mscale=1.1)
            q_out = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
            moeq4.moe_kv_append(cache, k, v, st, pt, spec, q, q_out)
            alone = torch.empty_like(q_out)
            moeq4.moe_rope(q, alone, pt, spec)
            assert torch.equal(q_out, alone)                    # one rotation, one set of bits
            turned = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device="cuda")
            moeq4.moe_rope(k, turned, pt, spec)
            moeq4.moe_kv_read(cache, st, k_out, None)
            want = O.bf16_value(O.to_bf16(quantised32(f64(turned), bits)))
            want[~kept] = 0
            assert np.array_equal(f64(k_out), want)
            ref = kv.rope(f64(q), pos, ph, rot, inter, 1.1)
            assert np.all(np.abs(f64(q_out) - ref) <= rope_bound(f64(q), ref, rot, inter, 1.1, 2.0 ** -8))
    here = q.clone()
    moeq4.moe_kv_append(cache, k, v, st, pt, spec, q, q)        # queries in place
    moeq4.moe_rope(here, here, pt, spec)
    assert torch.equal(q, here)
    assert moeq4.moe_get_device_error(cache) == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_append_of_unusual_values(bits):
    big = 3.0e38
    rows = np.zeros((8, 1, 64))
    rows[1] = -2.5                                   # constant: code 0, the bias alone
    rows[2, 0, 5] = np.nan
    rows[3, 0, 7] = np.inf
    rows[4, 0, :2] = (big, -big)                     # max - min passes the largest float
    rows[5, 0, 0] = 2.0 ** -120
    rows[6, 0, 3] = -np.inf
    rows[7] = np.linspace(-1, 1, 64)
    k = bf16_tensor(rows)
    cache = moeq4.KVCache.alloc(1, 16, 1, 64, bits)
    slots = torch.arange(8, dtype=torch.int32, device="cuda")
    out = torch.empty_like(k)
    moeq4.moe_kv_append(cache, k, k, slots)
    moeq4.moe_kv_read(cache, slots, out, None)
    got, x = f64(out), f64(k)
    for r in (2, 3, 6):
        assert np.all(np.isnan(got[r]))
    for r in (0, 1, 4, 5, 7):
        span = x[r].max() - x[r].min()
        step = span / (2 ** bits - 1)
        # a rounded code; the bf16 scale over all codes (span * 2^-8) and bf16 of the result
        assert np.all(np.abs(got[r] - x[r]) <= step * 0.5 + (span + np.abs(x[r])) * 2.0 ** -8)
    assert np.all(got[1] == -2.5) and np.all(got[0] == 0)


def test_slots_outside_the_cache_are_reported():
    cache = moeq4.KVCache.alloc(2, 16, 1, 64, 8)
    cache.data.zero_()
    k = torch.randn((3, 1, 64), device="cuda").bfloat16()
    slots = torch.tensor([-1, 32, -2], dtype=torch.int32, device="cuda")
    moeq4.moe_kv_append(cache, k, k, slots)
    assert moeq4.moe_get_device_error(cache) == moeq4.MOE_DEVERR_BAD_SLOT
    assert not cache.data.any()
    cache.err.zero_()
    out = torch.ones((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    moeq4.moe_kv_read(cache, slots[:1], out[:1], None)
    assert moeq4.moe_get_device_error(cache) == 0
    moeq4.moe_kv_read(cache, slots, out, None)
    assert moeq4.moe_get_device_error(cache) == moeq4.MOE_DEVERR_BAD_SLOT
    assert not out.any()


# ---------------------------------------------------------------- attention

class Case:
    """Contexts in shuffled pages of a cache whose unwritten bytes read as NaN."""

    def __init__(self, seed, lens, Hq, Hkv, D, bits, P, prefix=0, nq=1, spare=2, scale_k=1.0):
        rng = np.random.default_rng(seed)
        self.B, self.nq, self.Hq, self.D, self.bits, self.P = len(lens), nq, Hq, D, bits, P
        per = [-(-n // P) for n in lens]
        pre = -(-prefix // P)
        total = sum(per) + pre + spare
        order = rng.permutation(total)
        data = np.full((total, 2, Hkv, kv.head_bytes(P, D, bits)), 255, np.uint8)
        stride = max(1, max(per, default=0)) + 1
        table = np.full((self.B, stride), 0x7FFFFFFF, np.int32)     # never read past the lengths
        self.own, at = [], 0
        for b, n in enumerate(lens):
            pages = order[at:at + per[b]]
            at += per[b]
            table[b, :per[b]] = pages
            self.own.append(self._fill(rng, data, pages, n, Hkv, scale_k))
        pages = order[at:at + pre]
        self.shared = self._fill(rng, data, pages, prefix, Hkv, scale_k)
        self.q = O.bf16_value(O.to_bf16(rng.standard_normal((self.B * nq, Hq, D))))
        self.cache = moeq4.KVCache(torch.from_numpy(data).cuda(), P, Hkv, D, bits)
        self.table = torch.from_numpy(table).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.prefix, self.max_len = prefix, max(lens, default=0)
        self.ptable = torch.from_numpy(pages.astype(np.int32)).cuda() if prefix else None

    def _fill(self, rng, data, pages, n, Hkv, scale_k):
        x = rng.standard_normal((n, 2, Hkv, self.D))
        x[:, 0] *= scale_k
        x = O.bf16_value(O.to_bf16(x))
        slots = [int(pages[t // self.P]) * self.P + t % self.P for t in range(n)]
        for s, row in zip(slots, x):
            kv.write_row(data, s, self.P, *kv.quantise(row, self.bits))
        return kv.read_rows(data, slots, self.P, self.D, self.bits)

    def run(self, q=None, out=None, max_len=None, scale=None, stream=None):
        q = bf16_tensor(self.q) if q is None else q
        out = torch.full((self.B * self.nq, self.Hq, self.D), 5.0, dtype=torch.bfloat16,
                         device="cuda") if out is None else out
        m = self.max_len if max_len is None else max_len
        ws = moeq4.alloc_workspace(moeq4.moe_kv_attention_workspace_size(
            self.B, self.nq, self.Hq, self.cache.Hkv, self.D, m, self.prefix))
        ws.fill_(255)                                       # its contents do not matter
        moeq4.moe_kv_attention(q, self.cache, self.table, self.lens, m, out, ws, nq=self.nq,
                               prefix_table=self.ptable, prefix_len=self.prefix, scale=scale,
                               stream=stream)
        return out

    def check(self, out, scale=None):
        """Operands of the products may be rounded with relative error u = 2^-8 (bf16): keys
        shift a logit by at most d = u * reach, which moves every weight by a factor
        e^(+-2d); weights and values add 2u; exponentials, sums and partial results 2^-11.
        The output's own rounding is 2^-8."""
        scale = self.D ** -0.5 if scale is None else scale
        q = self.q.reshape(self.B, self.nq, self.Hq, self.D)
        ref, spread, reach = kv.attention(q, self.own, self.shared, scale)
        got = f64(out).reshape(ref.shape)
        u = 2.0 ** -8
        loose = np.expm1(2 * u * reach)[..., None] + 2 * u + 2.0 ** -11
        assert np.all(np.isfinite(got))
        assert np.all(np.abs(got - ref) <= u * np.abs(ref) + spread * loose + 1e-30)
        # and as a whole: bf16 rounds with 1.7e-3 in the mean square; outputs and operands together
        norm = np.linalg.norm(ref)
        assert np.linalg.norm(got - ref) <= 4e-3 * norm
        assert moeq4.moe_get_device_error(self.cache) == 0


LENS = {
    "one": [1], "block": [16], "past_block": [17], "ragged": [0, 1, 15, 16, 31, 33, 64, 130, 0],
    "long": [3001], "mixed": [700, 0, 5],
}


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", list(LENS))
def test_attention_lengths(lens, D, bits):
    c = Case(D + bits, LENS[lens], 8, 2, D, bits, 16)
    c.check(c.run())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (16, 2), (24, 4), (5, 1), (16, 1), (9, 3), (40, 2)])
def test_attention_head_groups(Hq, Hkv, bits):
    c = Case(Hq, [90, 0, 33], Hq, Hkv, 128, bits, 48)
    c.check(c.run())


@pytest.mark.parametrize("P", [16, 32, 48, 80, 128, 256, 4096])
def test_attention_page_sizes(P):
    for bits in (8, 4):
        c = Case(P, [P - 1, P, P + 1, 3] if P < 4096 else [300], 8, 2, 64, bits, P, prefix=70, spare=0)
        c.check(c.run())


@pytest.mark.parametrize("nq", [2, 3, 5, 8, 17, 64, 150])
@pytest.mark.parametrize("prefix", [0, 33])
def test_attention_several_query_tokens(nq, prefix):
    # lengths below nq: the first query tokens see no own token
    for bits, D in ((8, 128), (4, 64), (8, 256)):
        c = Case(nq, [nq, max(0, nq - 1), 0, 200, nq + 1], 4, 2, D, bits, 32, prefix=prefix, nq=nq)
        c.check(c.run())


@pytest.mark.parametrize("prefix", [1, 15, 16, 63, 64, 65, 127, 129, 1000])
@pytest.mark.parametrize("B,Hq,Hkv,D,bits", [(1, 4, 2, 64, 8), (3, 16, 2, 128, 4), (20, 8, 1, 256, 8),
                                             (9, 16, 1, 128, 8), (33, 8, 2, 64, 4)])
def test_attention_shared_prefix(prefix, B, Hq, Hkv, D, bits):
    lens = [(7 * b) % 40 for b in range(B)]
    c = Case(prefix + B, lens, Hq, Hkv, D, bits, 48, prefix=prefix)
    c.check(c.run())


def test_attention_prefix_with_no_own_tokens():
    c = Case(3, [0, 0, 0], 8, 2, 128, 8, 16, prefix=77)
    c.check(c.run())


def test_attention_sees_nothing():
    c = Case(4, [0, 0], 8, 2, 64, 8, 16)
    assert not c.run().any()
    assert not c.run(max_len=100000 // 16 * 0).any()
    e = torch.empty((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    moeq4.moe_kv_attention(e, c.cache, c.table[:0], c.lens[:0], 10, e, moeq4.alloc_workspace(256))


@pytest.mark.parametrize("scale_k,scale", [(30.0, None), (1e-3, None), (1.0, 0.0), (1.0, 2.0), (1.0, -0.1)])
def test_attention_sharp_and_flat_scores(scale_k, scale):
    # sharp scores: bounds grow with the logits' reach, so only their sharpest row is compared as a whole
    c = Case(11, [257, 40], 8, 2, 128, 8, 16, prefix=50, scale_k=scale_k)
    out = c.run(scale=scale)
    s = 128 ** -0.5 if scale is None else scale
    ref, spread, reach = kv.attention(c.q.reshape(2, 1, 8, 128), c.own, c.shared, s)
    u = 2.0 ** -8
    loose = np.expm1(np.minimum(2 * u * np.abs(reach), 50))[..., None] + 2 * u + 2.0 ** -11
    got = f64(out).reshape(ref.shape)
    assert np.all(np.abs(got - ref) <= u * np.abs(ref) + spread * loose + 1e-30)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 60])
def test_attention_values_far_from_one(size):
    # values (and keys, with the scale taking them back) of any magnitude keep their precision
    c = Case(12, [300, 2], 8, 2, 64, 4, 16, prefix=20)
    data = c.cache.data.cpu().numpy().copy()
    P, D = 16, 64
    words = data[..., P * 32:].reshape(*data.shape[:3], P, 2, 2).copy().view("<u2")[..., 0]
    val = O.bf16_value(words)
    fine = np.isfinite(val)
    words[fine] = O.to_bf16(val[fine] * size)
    data[..., P * 32:] = words.view(np.uint8).reshape(*data.shape[:3], -1)
    c.cache = moeq4.KVCache(torch.from_numpy(data).cuda(), P, 2, D, 4)
    mul = lambda kvs: (kvs[0] * size, kvs[1] * size)
    c.own, c.shared = [mul(o) for o in c.own], mul(c.shared)
    s = D ** -0.5 / size
    c.check(c.run(scale=s), s)


def test_attention_of_nonfinite_seen_rows():
    # a NaN that is seen spreads to its request's rows of that head, and nowhere else
    c = Case(13, [40, 40], 4, 2, 64, 8, 16)
    clean = c.run()
    k = torch.full((1, 2, 64), 0.5, device="cuda").bfloat16()
    k[:, 1] = float("nan")
    moeq4.moe_kv_append(c.cache, k, k, (c.table[1, 2:3] * 16 + 4).int())
    out = c.run()
    assert torch.equal(out[0], clean[0])
    assert torch.isfinite(out[1, :2]).all() and torch.isnan(out[1, 2:]).all()


def test_attention_strides_and_streams():
    c = Case(14, [300, 17, 0], 8, 2, 128, 8, 32, prefix=40, nq=2)
    want = c.run()
    c.check(want)
    wide = torch.full((6, 8 + 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = bf16_tensor(c.q)
    out = torch.full((8, 6, 136), 2.0, dtype=torch.bfloat16, device="cuda")
    view = out.transpose(0, 1)[..., :128]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(q=wide[:, 2:10], out=view)
    other = c.run(stream=side)
    side.synchronize()
    assert torch.equal(view, want) and torch.equal(other, want)
    assert (out[..., 128:] == 2).all()


def test_attention_repeats_bit_for_bit():
    c = Case(15, [2000, 3, 900], 16, 2, 128, 4, 64, prefix=500)
    a = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), a)


def test_attention_max_len_is_only_a_bound():
    c = Case(16, [70, 0, 300], 8, 2, 64, 8, 16)
    c.table = torch.cat((c.table, torch.full((3, 5000), 0x7FFFFFFF, dtype=torch.int32, device="cuda")), 1)
    c.check(c.run(max_len=80000))


def test_attention_bad_pages_and_lengths_are_reported():
    c = Case(17, [40, 40], 8, 2, 64, 8, 16, prefix=20)
    clean = c.run()
    keep = int(c.table[1, 1])
    c.table[1, 1] = c.cache.pages                        # tokens 16..31 of request 1 are left out
    out = c.run()
    assert moeq4.moe_get_device_error(c.cache) == moeq4.MOE_DEVERR_BAD_PAGE
    c.cache.err.zero_()
    assert torch.equal(out[0], clean[0])
    full = c.own[1]
    c.own[1] = tuple(np.concatenate((x[:16], x[32:])) for x in full)
    c.check(out)
    c.table[1, 1], c.own[1] = keep, full
    c.lens[0] = -3                                       # taken as no own tokens
    c.lens[1] = 41                                       # above max_len: taken as 40
    out = c.run()
    assert moeq4.moe_get_device_error(c.cache) == moeq4.MOE_DEVERR_BAD_LENGTH
    assert torch.equal(out[1], clean[1]) and torch.isfinite(out[0]).all()


def test_attention_and_write_past_four_gigabytes():
    # pages whose byte offset passes 2^32 (page 2100 of 2 MB pages is at 4.4 GB)
    Hkv, D, P = 8, 128, 1024
    cache = moeq4.KVCache.alloc(2102, P, Hkv, D, 8)
    assert cache.data.numel() > 2 ** 32
    cache.data.fill_(255)
    rng = np.random.default_rng(18)
    n = 40
    k = bf16_tensor(rng.standard_normal((n, Hkv, D)))
    slots = (2100 * P + torch.arange(n, device="cuda")).int()
    moeq4.moe_kv_append(cache, k, k, slots)
    back = torch.empty_like(k)
    moeq4.moe_kv_read(cache, slots, None, back)
    assert np.array_equal(f64(back), O.bf16_value(O.to_bf16(quantised32(f64(k), 8))))
    near = moeq4.KVCache.alloc(1, P, Hkv, D, 8)
    near.data.copy_(cache.data.view(2102, -1)[2100])
    q = bf16_tensor(rng.standard_normal((1, 16, D)))
    outs = []
    for ca, page in ((cache, 2100), (near, 0)):
        table = torch.tensor([[page]], dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)
        ws = moeq4.alloc_workspace(moeq4.moe_kv_attention_workspace_size(1, 1, 16, Hkv, D, n, n))
        moeq4.moe_kv_attention(q, ca, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n,
                               out, ws, prefix_table=table[0], prefix_len=n)
        outs.append(out)
    assert torch.equal(*outs) and torch.isfinite(outs[0]).all()


def test_calls_replay_in_a_graph():
    c = Case(19, [100, 37], 8, 2, 128, 8, 16, prefix=64)
    want = c.run()
    q, out = bf16_tensor(c.q), torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    ws = moeq4.alloc_workspace(moeq4.moe_kv_attention_workspace_size(2, 1, 8, 2, 128, 100, 64))
    go = lambda: moeq4.moe_kv_attention(q, c.cache, c.table, c.lens, 100, out, ws,
                                        prefix_table=c.ptable, prefix_len=64)
    go()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    out.zero_()
    g.replay()
    assert torch.equal(out, want)
