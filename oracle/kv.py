"""CPU oracle of the attention side: rotary positions, the quantised key/value
cache and attention over it. Plain numpy in float64, sharing nothing with the
product path.

Rotary positions: pair i of the first ``rot`` elements ((i, i + rot/2), or
(2i, 2i + 1) when interleaved) is turned by 2 pi frac(pos * phase_i / 2^64).
Cache: groups of 64 elements along a head share a bf16 scale and bias, value =
scale * code + bias (the same groupwise-affine format as the expert weights,
with 8- or 4-bit codes). Attention: softmax over the shared prefix and the
request's own tokens, causal among its query tokens; a row that sees nothing
is zero.
"""
from __future__ import annotations

import numpy as np

from . import bf16_value, to_bf16

GROUP = 64


def rope(x, pos, phase, rot, interleaved=False, mscale=1.0, backward=False):
    """x [T][H][D] turned, float64."""
    with np.errstate(over="ignore"):
        w = np.asarray(pos, dtype=np.int64).astype(np.uint64)[:, None] * np.asarray(phase, np.uint64)[None]
    angle = 2.0 * np.pi * (w.astype(np.float64) / 2.0 ** 64)
    c, s = np.cos(angle)[:, None] * mscale, np.sin(angle)[:, None] * mscale
    if backward:
        s = -s
    y = np.array(x, dtype=np.float64)
    a, b = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
            else (slice(0, rot // 2), slice(rot // 2, rot)))
    xa, xb = y[..., a].copy(), y[..., b].copy()
    y[..., a] = xa * c - xb * s
    y[..., b] = xb * c + xa * s
    return y


def quantise(x, bits):
    """x [...][D] (bf16 values) -> codes uint8 [...][D], scale and bias [...][D/64] (bf16 values)."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = g.min(-1), g.max(-1)
    levels = 2 ** bits - 1
    scale = bf16_value(to_bf16((hi - lo) / levels))
    safe = np.where(scale > 0, scale, 1.0)
    code = np.clip(np.rint((g - lo[..., None]) / safe[..., None]), 0, levels)
    code = np.where(scale[..., None] > 0, code, 0)
    return code.reshape(x.shape).astype(np.uint8), scale, lo


def values(code, scale, bias):
    g = code.astype(np.float64).reshape(*code.shape[:-1], -1, GROUP)
    return (g * scale[..., None] + bias[..., None]).reshape(code.shape)


def head_bytes(page_size, D, bits):
    return page_size * (D * bits // 8 + D // GROUP * 4)


def write_row(data, slot, page_size, code, scale, bias):
    """One token of the cache bytes data [pages][2][Hkv][head_bytes]: code [2][Hkv][D] etc."""
    D = code.shape[-1]
    hb = data.shape[-1]
    bits = 8 if hb == head_bytes(page_size, D, 8) else 4
    page, r = divmod(int(slot), page_size)
    rb, nb = D * bits // 8, D // GROUP
    packed = code if bits == 8 else (code[..., 0::2] | (code[..., 1::2] << 4))
    data[page, :, :, r * rb:(r + 1) * rb] = packed
    words = np.stack((to_bf16(scale), to_bf16(bias)), -1).astype("<u2")
    at = page_size * rb + r * nb * 4
    data[page, :, :, at:at + nb * 4] = words.reshape(*words.shape[:2], -1).view(np.uint8)


def read_rows(data, slots, page_size, D, bits):
    """keys, values [n][Hkv][D] float64 of the listed slots."""
    rb, nb = D * bits // 8, D // GROUP
    out = []
    for slot in slots:
        page, r = divmod(int(slot), page_size)
        raw = data[page, :, :, r * rb:(r + 1) * rb]
        code = raw if bits == 8 else np.stack((raw & 15, raw >> 4), -1).reshape(*raw.shape[:2], D)
        at = page_size * rb + r * nb * 4
        words = np.ascontiguousarray(data[page, :, :, at:at + nb * 4]).view("<u2")
        words = bf16_value(words.reshape(*words.shape[:2], nb, 2).astype(np.uint16))
        out.append(values(code, words[..., 0], words[..., 1]))
    a = np.stack(out) if out else np.zeros((0, 2, data.shape[2], D))
    return a[:, 0], a[:, 1]


def attention(q, own, shared, scale):
    """q [B][nq][Hq][D]; own: per request (keys, values) [n][Hkv][D]; shared: the prefix's.

    Returns (o, spread, reach): the output; sum_t p_t |v_t| per element; and the largest
    scale * sum_d |q_d| |k_td| of each row's seen tokens (for error bounds)."""
    B, nq, Hq, D = q.shape
    o, spread = np.zeros(q.shape), np.zeros(q.shape)
    reach = np.zeros((B, nq, Hq))
    for b in range(B):
        k = np.concatenate((shared[0], own[b][0]))
        v = np.concatenate((shared[1], own[b][1]))
        n, pre = len(own[b][0]), len(shared[0])
        G = Hq // k.shape[1]
        for i in range(nq):
            seen = pre + max(0, n - nq + 1 + i)
            if not seen:
                continue
            for h in range(Hq):
                kh, vh = k[:seen, h // G], v[:seen, h // G]
                z = scale * (kh @ q[b, i, h])
                p = np.exp(z - z.max())
                p /= p.sum()
                o[b, i, h] = p @ vh
                spread[b, i, h] = p @ np.abs(vh)
                reach[b, i, h] = scale * (np.abs(kh) @ np.abs(q[b, i, h])).max()
    return o, spread, reach
