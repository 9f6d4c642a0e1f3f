"""Command-line drivers of single library calls on the seeded synthetic inputs,
for profilers (ncu) and quick timings.

    python -m routing_q4_grouped_gb300.drivers layer  T [calls]   # moe_layer, full-width layer
    python -m routing_q4_grouped_gb300.drivers router T [calls]   # moe_router_topk
    python -m routing_q4_grouped_gb300.drivers attention B nq length prefix [bits] [D] [calls]
                                                                  # moe_kv_attention
    python -m routing_q4_grouped_gb300.drivers step B length [bits] [calls]   # one decoder step

The full-width layer has d = 2048, 256 experts, top-8, f = f_s = 512 and the
value recipe of the t512 workload; T tokens of its seeded x and logits. Each
call goes through the C-ABI on the current stream; the driver prints the mean
time of the calls after the first (CUDA events) and the device error word.

``attention``: B requests with nq query tokens each over contexts of `length`
tokens behind a shared prefix (0: none), 16 query and 2 key/value heads.

``step`` runs the attention side and the expert layer together, as one decoder
layer uses them for a batch of B requests that decode one token each: the fused
query/key/value projection, moe_kv_append (turn, quantise, write),
moe_kv_attention, the output projection, then moe_layer on the sum. The two
projections are plain matrix products of random bf16 weights.
"""
from __future__ import annotations

import dataclasses
import sys

import numpy as np
import torch

from . import moeq4, synth


def _layer(T: int, calls: int) -> None:
    cfg = dataclasses.replace(synth.CONFIGS["t512"], T=T)
    W = moeq4.DeviceWeights.from_host(synth.gen_weights(cfg, 0))
    x = torch.from_numpy(synth.gen_x(cfg, T).view(np.int16)).cuda().view(torch.bfloat16)
    lg = torch.from_numpy(synth.gen_logits(cfg, 0, T)).cuda()
    lay = moeq4.Layer(W, T, cfg.k, None)
    _timed(lambda: lay(x, lg), calls, lay.route)


def _router(T: int, calls: int) -> None:
    cfg = dataclasses.replace(synth.CONFIGS["t4096"], T=T)
    x = torch.from_numpy(synth.gen_x(cfg, T).view(np.int16)).cuda().view(torch.bfloat16)
    wr = torch.from_numpy(synth.gen_router(cfg).view(np.int16)).cuda().view(torch.bfloat16)
    out = moeq4.RouteBuffers.alloc(T, cfg.E, cfg.k, 128)
    lg = torch.empty((T, cfg.E), dtype=torch.float32, device="cuda")
    _timed(lambda: moeq4.moe_router_topk(x, wr, out, lg), calls, out)


HQ, HKV = 16, 2


def _cache(pages: int, bits: int, D: int, page_size: int = 64) -> moeq4.KVCache:
    """A cache whose every slot holds a quantised normal row."""
    cache = moeq4.KVCache.alloc(pages, page_size, HKV, D, bits)
    for p in range(0, pages, 512):
        n = min(512, pages - p) * page_size
        kv = torch.randn((n, 2 * HKV, D), device="cuda").bfloat16()
        slots = torch.arange(p * page_size, p * page_size + n, dtype=torch.int32, device="cuda")
        moeq4.moe_kv_append(cache, kv[:, :HKV], kv[:, HKV:], slots)
    return cache


def _tables(B: int, length: int, prefix: int, page_size: int = 64):
    per, pre = -(-length // page_size), -(-prefix // page_size)
    order = torch.randperm(B * per + pre, device="cuda").int()
    return B * per + pre, order[:B * per].view(B, per).contiguous(), order[B * per:]


def _attention(B: int, nq: int, length: int, prefix: int, bits: int, D: int, calls: int) -> None:
    pages, table, ptable = _tables(B, length, prefix)
    cache = _cache(pages, bits, D)
    q = torch.randn((B * nq, HQ, D), device="cuda").bfloat16()
    out = torch.empty_like(q)
    lens = torch.full((B,), length, dtype=torch.int32, device="cuda")
    ws = moeq4.alloc_workspace(moeq4.moe_kv_attention_workspace_size(B, nq, HQ, HKV, D, length, prefix))
    _timed(lambda: moeq4.moe_kv_attention(q, cache, table, lens, length, out, ws, nq=nq,
                                          prefix_table=ptable, prefix_len=prefix), calls, cache)


def _step(B: int, length: int, bits: int, calls: int) -> None:
    cfg = dataclasses.replace(synth.CONFIGS["t512"], T=B)
    D = cfg.d // HQ
    W = moeq4.DeviceWeights.from_host(synth.gen_weights(cfg, 0))
    lay = moeq4.Layer(W, B, cfg.k, None)
    lg = torch.from_numpy(synth.gen_logits(cfg, 0, B)).cuda()
    x = torch.from_numpy(synth.gen_x(cfg, B).view(np.int16)).cuda().view(torch.bfloat16)
    w_qkv = torch.randn((cfg.d, (HQ + 2 * HKV) * D), device="cuda").mul_(cfg.d ** -0.5).bfloat16()
    w_out = torch.randn((HQ * D, cfg.d), device="cuda").mul_(cfg.d ** -0.5).bfloat16()
    pages, table, _ = _tables(B, length, 0)
    cache = _cache(pages, bits, D)
    rope = moeq4.RopeSpec(moeq4.moe_rope_phases(D, 1e6).cuda(), D)
    lens = torch.full((B,), length, dtype=torch.int32, device="cuda")
    pos = lens - 1                                     # the new token is the context's last
    last = (pos // cache.page_size).long()
    slots = (table.gather(1, last[:, None])[:, 0] * cache.page_size + pos % cache.page_size).int()
    att = torch.empty((B, HQ, D), dtype=torch.bfloat16, device="cuda")
    ws = moeq4.alloc_workspace(moeq4.moe_kv_attention_workspace_size(B, 1, HQ, HKV, D, length, 0))

    def step():
        qkv = (x @ w_qkv).view(B, HQ + 2 * HKV, D)
        q = qkv[:, :HQ]
        moeq4.moe_kv_append(cache, qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], slots, pos, rope, q, q)
        moeq4.moe_kv_attention(q, cache, table, lens, length, att, ws)
        h = x + att.view(B, -1) @ w_out
        return lay(h, lg)

    _timed(step, calls, cache)
    if moeq4.moe_get_device_error(lay.route):
        raise RuntimeError("device error word of the expert layer set")


def _timed(fn, calls: int, route) -> None:
    fn()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(calls - 1):
        fn()
    e1.record()
    torch.cuda.synchronize()
    us = e0.elapsed_time(e1) / max(1, calls - 1) * 1e3
    print(f"mean {us:.1f} us per call over {calls - 1} calls; device error word "
          f"{moeq4.moe_get_device_error(route)}")


def main(argv) -> None:
    what, nums = argv[1], [int(v) for v in argv[2:]]
    if what == "attention":
        B, nq, length, prefix, bits, D, calls = nums + [8, 128, 4][len(nums) - 4:]
        _attention(B, nq, length, prefix, bits, D, calls)
    elif what == "step":
        B, length, bits, calls = nums + [8, 4][len(nums) - 2:]
        _step(B, length, bits, calls)
    else:
        {"layer": _layer, "router": _router}[what](nums[0], nums[1] if len(nums) > 1 else 4)


if __name__ == "__main__":
    main(sys.argv)
