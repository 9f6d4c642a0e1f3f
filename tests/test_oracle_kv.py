"""The attention-side oracle against closed forms and brute force, and the host
side of the calls: frequencies, sizes and refusals."""
import ctypes
import math
import os

import numpy as np
import pytest

import oracle as O
from oracle import kv


@pytest.fixture(scope="module")
def L():
    from routing_q4_grouped_gb300 import build, moeq4
    if not os.path.exists(moeq4.LIB_PATH):
        build.build()
    return moeq4


def _phase(rot, base=10000.0):
    f = base ** (-2.0 * np.arange(rot // 2) / rot) / (2 * math.pi)
    return np.array([int(math.ldexp(x, 64)) for x in f], dtype=np.uint64)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_rotation_by_the_position(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 12))
    ph = _phase(8)
    y = kv.rope(x, [0, 5, -7], ph, 8, interleaved)
    assert np.array_equal(y[0], x[0])                       # position 0
    assert np.array_equal(y[..., 8:], x[..., 8:])           # elements past rot
    z = x[1, 0, :8].reshape(4, 2).T if interleaved else x[1, 0, :8].reshape(2, 4)
    w = (z[0] + 1j * z[1]) * np.exp(1j * 5 * 10000.0 ** (-np.arange(4) / 4.0))
    w = np.stack((w.real, w.imag))
    assert np.allclose(y[1, 0, :8], (w.T if interleaved else w).reshape(-1), atol=1e-13)
    # the transposed rotation undoes it, and is the gradient: <R x, g> = <x, R^T g>
    back = kv.rope(y, [0, 5, -7], ph, 8, interleaved, backward=True)
    assert np.allclose(back, x, atol=1e-13)
    g = rng.standard_normal(x.shape)
    lhs = (kv.rope(x, [9, 9, 9], ph, 8, interleaved, 1.3) * g).sum()
    rhs = (x * kv.rope(g, [9, 9, 9], ph, 8, interleaved, 1.3, True)).sum()
    assert abs(lhs - rhs) < 1e-12 * abs(lhs) + 1e-12


def test_rope_scores_depend_on_distance_only_at_long_positions():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    ph = _phase(64)
    dot = lambda a, b: float((kv.rope(q, [a], ph, 64) * kv.rope(k, [b], ph, 64)).sum())
    assert abs(dot(3, 10) - dot(2 ** 30 + 3, 2 ** 30 + 10)) < 1e-9


@pytest.mark.parametrize("bits", [8, 4])
def test_quantised_values_stay_within_a_step(bits):
    rng = np.random.default_rng(bits)
    x = O.bf16_value(O.to_bf16(rng.standard_normal((5, 3, 128)) * 3))
    code, scale, bias = kv.quantise(x, bits)
    err = np.abs(kv.values(code, scale, bias) - x).reshape(5, 3, 2, 64).max(-1)
    # half a step of rounding, plus the last codes where the rounded scale falls short
    assert np.all(err <= scale * (0.5 + (2 ** bits - 1) * 2.0 ** -8) * (1 + 1e-9))
    code, scale, bias = kv.quantise(np.full((1, 64), -1.5), bits)
    assert np.all(kv.values(code, scale, bias) == -1.5)


@pytest.mark.parametrize("bits", [8, 4])
def test_cache_rows_round_trip(bits):
    rng = np.random.default_rng(bits)
    P, H, D = 16, 3, 128
    data = np.full((4, 2, H, kv.head_bytes(P, D, bits)), 255, np.uint8)
    x = O.bf16_value(O.to_bf16(rng.standard_normal((2, 2, H, D))))
    for slot, row in zip((37, 5), x):
        kv.write_row(data, slot, P, *kv.quantise(row, bits))
    k, v = kv.read_rows(data, [5, 37], P, D, bits)
    ref = np.stack([kv.values(*kv.quantise(row, bits)) for row in x])
    assert np.array_equal(k, ref[::-1, 0]) and np.array_equal(v, ref[::-1, 1])


def test_attention_closed_forms():
    rng = np.random.default_rng(3)
    none = (np.zeros((0, 1, 64)),) * 2
    k, v = rng.standard_normal((6, 1, 64)), rng.standard_normal((6, 1, 64))
    q = rng.standard_normal((1, 2, 2, 64))
    # equal keys: the mean of the seen values; 6 tokens, 2 query tokens
    o, _, _ = kv.attention(q, [(np.zeros_like(k), v)], none, 1.0)
    assert np.allclose(o[0, 0, 0], v[:5, 0].mean(0)) and np.allclose(o[0, 1, 1], v[:, 0].mean(0))
    # a split into prefix and own tokens changes nothing where both are seen whole
    a, _, _ = kv.attention(q[:, 1:], [(k, v)], none, 0.3)
    b, _, _ = kv.attention(q[:, 1:], [(k[4:], v[4:])], (k[:4], v[:4]), 0.3)
    assert np.allclose(a, b)
    # one token with two queries: the first sees nothing
    o, _, _ = kv.attention(q, [(k[:1], v[:1])], none, 1.0)
    assert np.all(o[0, 0] == 0) and np.allclose(o[0, 1, 0], v[0, 0])


@pytest.mark.parametrize("scaling,factor", [(0, 1.0), (1, 4.0), (2, 8.0), (3, 16.0)])
@pytest.mark.parametrize("rot,base", [(128, 1e4), (64, 1e6), (24, 5e5)])
def test_frequencies(L, scaling, factor, rot, base):
    ph = L.moe_rope_phases(rot, base, scaling, factor, trained=4096, fast=32, slow=1)
    got = ph.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    i = np.arange(rot // 2)
    b = base * factor ** (rot / (rot - 2)) if scaling == 2 else base
    f = b ** (-2.0 * i / rot)
    if scaling == 1:
        f /= factor
    # double precision throughout (pow to an ulp or two), then a 64-bit fraction of a turn
    close = dict(rtol=1e-14, atol=2 * math.pi * 2.0 ** -64)
    if scaling == 3:
        turns = 4096 * f / (2 * math.pi)
        assert np.allclose(got[turns >= 33], f[turns >= 33], **close)
        low = turns * f[0] <= 0.6
        assert np.allclose(got[low], f[low] / factor, **close)
        slack = f * close["rtol"] + close["atol"]
        assert np.all(got <= f + slack) and np.all(got >= f / factor - slack)
        return
    assert np.allclose(got, f, **close)


def test_frequencies_refused(L):
    bad = [dict(rot=3), dict(rot=0), dict(base=1.0), dict(base=float("nan")), dict(factor=0.5),
           dict(scaling=4), dict(scaling=-1), dict(scaling=3, trained=0.0),
           dict(scaling=3, trained=10.0, fast=1.0, slow=2.0), dict(scaling=2, rot=2)]
    for b in bad:
        with pytest.raises(L.MoeError):
            L.moe_rope_phases(**{**dict(rot=64, base=1e4), **b})


def test_cache_sizes(L):
    assert L.moe_kv_cache_size(3, 16, 2, 128, 8) == 3 * 2 * 2 * 16 * (128 + 8)
    assert L.moe_kv_cache_size(100000, 256, 8, 256, 4) == 100000 * 2 * 8 * 256 * (128 + 16)
    for bad in [(0, 16, 2, 128, 8), (1, 8, 2, 128, 8), (1, 24, 2, 128, 8), (1, 8192, 2, 128, 8),
                (1, 16, 0, 128, 8), (1, 16, 2, 96, 8), (1, 16, 2, 128, 16),
                (2 ** 27, 16, 1, 64, 4)]:
        assert L.moe_kv_cache_size(*bad) == 0, bad


FAKE = 1 << 20      # aligned non-null, never dereferenced: every call below is refused first


def _cache(L, **kw):
    f = dict(data=FAKE, err=FAKE, pages=4, page_size=16, Hkv=2, D=128, bits=8)
    f.update(kw)
    return L.KVCacheC(f["data"], f["err"], f["pages"], f["page_size"], f["Hkv"], f["D"], f["bits"])


def test_rope_arguments_rejected_on_host(L):
    lib = L.lib()

    def call(x=FAKE, xr=256, xh=128, o=FAKE, orow=256, oh=128, pos=FAKE, T=4, H=2, D=128, phase=FAKE,
             rot=128, inter=0, m=1.0, back=0, dtype=0):
        spec = L.RopeSpecC(phase, rot, inter, m)
        return lib.moe_rope(x, xr, xh, o, orow, oh, pos, T, H, D, ctypes.byref(spec), back, dtype, None)
    assert call(T=0) == 0
    assert call(x=None) == call(o=None) == call(pos=None) == call(phase=None) == -1
    assert call(T=-1) == call(H=0) == call(back=2) == call(dtype=3) == call(inter=2) == -1
    assert call(m=float("nan")) == -1
    assert call(rot=130) == call(rot=3) == call(rot=0) == call(D=127) == -2
    assert call(xr=-256) == -2
    assert call(o=2 * FAKE, orow=128) == -2              # output rows overlap
    assert call(o=2 * FAKE, orow=256, oh=64) == -2       # output heads overlap
    assert call(orow=512) == -1                          # in place with other strides
    assert call(x=FAKE + 1) == call(pos=FAKE + 2) == call(phase=FAKE + 4) == -7
    assert lib.moe_rope(FAKE, 256, 128, FAKE, 256, 128, FAKE, 4, 2, 128, None, 0, 0, None) == -1


def test_append_and_read_arguments_rejected_on_host(L):
    lib = L.lib()
    spec = L.RopeSpecC(FAKE, 128, 0, 1.0)

    def call(cache=None, rope=spec, **kw):
        a = L.KVNewC(FAKE, 256, 128, FAKE, 256, 128, FAKE, 512, 128, FAKE, 512, 128, FAKE, FAKE,
                     ctypes.pointer(rope) if rope else None, 4, 4)
        for n, v in kw.items():
            setattr(a, n, v)
        return lib.moe_kv_append(ctypes.byref(a), ctypes.byref(cache or _cache(L)), None)
    assert call(T=0) == 0
    assert call(k=None) == call(v=None) == call(slots=None) == call(pos=None) == call(q_out=None) == -1
    assert call(T=-1) == call(Hq=0) == call(rope=None) == -1        # queries need a rotation
    assert call(k_row=-8) == call(q_head=-8) == call(qo_row=128) == -2
    assert call(k=FAKE + 2) == call(v_row=257) == call(q_head=4) == call(slots=FAKE + 2) == -7
    assert call(qo_row=1024) == -1                                   # in place with other strides
    assert call(rope=L.RopeSpecC(FAKE, 130, 0, 1.0)) == -2
    for bad, want in ((dict(data=None), -1), (dict(err=None), -1), (dict(pages=0), -2),
                      (dict(page_size=20), -2), (dict(D=80), -2), (dict(bits=2), -2),
                      (dict(data=FAKE + 8), -7), (dict(err=FAKE + 2), -7)):
        assert call(_cache(L, **bad)) == want, bad
        assert lib.moe_kv_read(ctypes.byref(_cache(L, **bad)), FAKE, 4, FAKE, FAKE, None) == want
    read = lambda s, n, k, v: lib.moe_kv_read(ctypes.byref(_cache(L)), s, n, k, v, None)
    assert read(FAKE, 0, None, None) == 0
    assert read(None, 4, FAKE, FAKE) == read(FAKE, -1, FAKE, FAKE) == read(FAKE, 4, None, None) == -1
    assert read(FAKE, 4, FAKE + 8, None) == read(FAKE + 1, 4, FAKE, None) == -7
    assert lib.moe_kv_append(None, ctypes.byref(_cache(L)), None) == -1
    assert lib.moe_kv_read(None, FAKE, 4, FAKE, FAKE, None) == -1


def test_attention_arguments_rejected_on_host(L):
    lib = L.lib()

    def call(cache=None, ws=FAKE, n=1 << 40, **kw):
        a = L.KVAttnC(FAKE, 512, 128, FAKE, 512, 128, FAKE, FAKE, FAKE, 4, 1, 4, 8, 100, 30, 0.1)
        for name, v in kw.items():
            setattr(a, name, v)
        return lib.moe_kv_attention(ctypes.byref(a), ctypes.byref(cache or _cache(L)), ws, n, None)
    assert call(B=0) == 0
    for kw in (dict(q=None), dict(out=None), dict(lens=None), dict(table=None), dict(ws=None),
               dict(prefix_table=None), dict(B=-1), dict(nq=0), dict(Hq=0), dict(max_len=-1),
               dict(prefix_len=-1), dict(scale=float("inf")), dict(table_stride=-1)):
        assert call(**kw) == -1, kw
    for kw in (dict(Hq=3), dict(table_stride=6), dict(q_row=-512), dict(out_row=128),
               dict(out_head=64), dict(B=1 << 30), dict(prefix_len=(1 << 30) + 1),
               dict(max_len=(1 << 30) + 1, table_stride=1 << 30)):
        assert call(**kw) == -2, kw
    for kw in (dict(q=FAKE + 8), dict(out=FAKE + 2), dict(ws=FAKE + 4), dict(lens=FAKE + 1),
               dict(table=FAKE + 2), dict(prefix_table=FAKE + 2), dict(q_row=513), dict(out_head=129,
               out_row=1032)):
        assert call(**kw) == -7, kw
    assert call(n=8) == -3
    assert call(_cache(L, D=80)) == -2
    assert lib.moe_kv_attention(None, ctypes.byref(_cache(L)), FAKE, 1 << 40, None) == -1


def test_binding_refuses_wrong_tensors(L):
    import torch
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="moe_rope: x must be .* CUDA tensor"):
        L.moe_rope(x, x, None, None)
    with pytest.raises(ValueError, match="bfloat16, float16 or float32"):
        L.moe_rope(x.double(), x, None, None)
    with pytest.raises(ValueError, match="KVCache: data must be a contiguous torch.uint8 CUDA"):
        L.KVCache(torch.zeros(64, dtype=torch.uint8), 16, 2, 128, 8)
    with pytest.raises(ValueError, match="sizes not allowed"):
        L.KVCache.alloc(4, 17, 2, 128, 8)
    with pytest.raises(ValueError, match="RopeSpec: phase"):
        L.RopeSpec(torch.zeros(64, dtype=torch.int64), 128)
