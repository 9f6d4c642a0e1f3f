"""Groups whose bf16 scale is below the smallest normal number."""
import numpy as np
import pytest
import torch

import oracle as O
from kv_case import Case
from routing_q4_grouped_gb300 import moeq4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 4])
def test_write_keeps_tiny_groups(bits):
    exps = list(range(-110, -129, -1))
    rows = np.stack([np.linspace(-0.3, 1.0, 64) * 2.0 ** e for e in exps])
    rows = np.concatenate((rows, np.stack([np.where(np.arange(64) % 3, 2.0 ** e, 0.0) for e in exps])))
    x = O.bf16_value(O.to_bf16(rows.astype(np.float32))).astype(np.float64)
    k = torch.from_numpy(x.astype(np.float32)).cuda().bfloat16().view(-1, 1, 64)
    n = k.shape[0]
    cache = moeq4.KVCache.alloc(4, 16, 1, 64, bits)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    out = torch.empty_like(k)
    moeq4.moe_kv_append(cache, k, k, slots)
    moeq4.moe_kv_read(cache, slots, out, None)
    got = out.double().cpu().numpy()[:, 0]
    for r in range(n):
        span = x[r].max() - x[r].min()
        step = span / (2 ** bits - 1)
        # a rounded code; the scale's rounding (2^-8 of it, or half of bf16's smallest number)
        # over all codes; the result's rounding
        bound = step * 0.5 * (1 + 2.0 ** -8) + (span + np.abs(x[r])) * 2.0 ** -8 \
            + (2 ** bits - 1) * 2.0 ** -134 + 2.0 ** -134
        assert np.all(np.abs(got[r] - x[r]) <= bound), (r, got[r], x[r])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("size", [2.0 ** -116, 2.0 ** -122])
@pytest.mark.parametrize("lens,nq,G", [([17, 40, 1], 1, 4), ([900, 65, 300], 9, 3)])
def test_attention_over_tiny_values(lens, nq, G, size, D, bits):
    # scales around and below 2^-126; outputs stay above it but for a few
    def shape(x, what, b):
        x[:, 1] *= size
    c = Case(D + bits, lens, 2 * G, 2, D, bits, 16, nq=nq, shape=shape)
    c.check(c.run(), norm=4e-3)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("size", [2.0 ** -112, 2.0 ** -116])
def test_many_rows_over_tiny_values(size, D, bits):
    # 560 rows a request: the kernel for many rows
    def shape(x, what, b):
        x[:, 1] *= size
    c = Case(D + bits, [2000, 65], 16, 2, D, bits, 16, nq=70, shape=shape)
    assert c.rows_kernel() == 2
    c.check(c.run(), norm=4e-3)
