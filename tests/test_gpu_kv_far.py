"""Caches and contexts whose page numbers pass 2^24."""
import pytest
import torch

from routing_q4_grouped_gb300 import moeq4

pytestmark = pytest.mark.gpu


def test_write_and_read_past_2_to_24_pages():
    P, D = 16, 64
    far = 2 ** 24
    cache = moeq4.KVCache.alloc(far + 8, P, 1, D, 4)         # 19.3 GB
    pages = cache.data.view(far + 8, -1)
    pages[:8].fill_(255)
    pages[far - 4:].fill_(255)
    near = moeq4.KVCache.alloc(8, P, 1, D, 4)
    near.data.fill_(255)
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = torch.randn((40, 2, D), generator=g, device="cuda").bfloat16()
    k, v = kv[:, :1], kv[:, 1:]
    at = torch.arange(40, dtype=torch.int32, device="cuda") + 17      # pages 1 .. 3
    moeq4.moe_kv_append(cache, k, v, at + far * P)
    moeq4.moe_kv_append(near, k, v, at)
    assert torch.equal(pages[far:], near.data.view(8, -1))
    assert (pages[:8] == 255).all() and (pages[far - 4:far] == 255).all()
    outs = [torch.empty((40, 1, D), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    moeq4.moe_kv_read(cache, at + far * P, outs[0], outs[1])
    moeq4.moe_kv_read(near, at, outs[2], outs[3])
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    assert moeq4.moe_get_device_error(cache) == 0


@pytest.mark.parametrize("Hq", [1, 64])                      # few query rows, and the kernel for many
def test_attention_past_2_to_28_tokens(Hq):
    # every page of the context is page 0 (keys and values 0: logits 0) but the last two,
    # whose keys give logits of 50: e^50 against 2^28 tokens of e^0, so the outputs are the
    # mean of their values
    P, D, n = 16, 64, 2 ** 28 + 32
    cache = moeq4.KVCache.alloc(3, P, 1, D, 8)
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.zeros((48, 1, D), device="cuda")
    k[16:] = 50.0 / 8.0
    v = torch.randn((48, 1, D), generator=g, device="cuda")
    v[:16] = 0
    slots = torch.arange(48, dtype=torch.int32, device="cuda")
    moeq4.moe_kv_append(cache, k.bfloat16(), v.bfloat16(), slots)
    back = torch.empty((48, 1, D), dtype=torch.bfloat16, device="cuda")
    moeq4.moe_kv_read(cache, slots, None, back)
    want = back[16:].double().mean(0)
    table = torch.zeros((1, n // P), dtype=torch.int32, device="cuda")
    table[0, -2], table[0, -1] = 1, 2
    q = torch.ones((1, Hq, D), device="cuda").bfloat16()
    out = torch.empty_like(q)
    ws = moeq4.alloc_workspace(moeq4.moe_kv_attention_workspace_size(1, 1, Hq, 1, D, n))
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    moeq4.moe_kv_attention(q, cache, table, lens, n, out, ws)
    # 32 equal weights; values rounded to bf16 (2^-9 of numbers up to 4) and the output's rounding
    assert (out.double() - want).abs().max() <= 4 * 2.0 ** -9 + 2.0 ** -8 * want.abs().max()
    assert moeq4.moe_get_device_error(cache) == 0
