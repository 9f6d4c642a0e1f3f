"""Command-line drivers of single library calls on the seeded synthetic inputs,
for profilers (ncu) and quick timings.

    python -m routing_q4_grouped_gb300.drivers layer  T [calls]   # moe_layer, full-width layer
    python -m routing_q4_grouped_gb300.drivers router T [calls]   # moe_router_topk
    python -m routing_q4_grouped_gb300.drivers attention B nq length prefix [bits] [D] [calls]
                                                                  # moe_kv_attention
    python -m routing_q4_grouped_gb300.drivers step B length [bits] [calls]   # one decoder step
    python -m routing_q4_grouped_gb300.drivers block B length [bits] [calls]  # ... from hidden rows
    python -m routing_q4_grouped_gb300.drivers linear T N K [e4m3] [calls]    # moe_linear
    python -m routing_q4_grouped_gb300.drivers norm T D [codes] [calls]       # moe_rms_norm
    python -m routing_q4_grouped_gb300.drivers scored T E groups [calls]      # moe_route_scored

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

``block`` is the step from one hidden row per request to the next: moe_rms_norm
with the residual, the projection, the norm of query and key heads, append,
attention, the output projection, moe_rms_norm, the router's logits, and
moe_layer_scored (sigmoid scores, a bias, 4 of 8 groups of experts).

``linear``: e4m3 0 or 1. ``norm``: rows with a residual, into bf16 or (codes 1) e4m3
codes. ``scored``: sigmoid scores with a bias, half of the groups, top 8.
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


class _Attention:
    """The attention side of one decoder layer for B requests that decode one token each."""

    def __init__(self, cfg, B: int, length: int, bits: int):
        self.B, self.length, self.D = B, length, cfg.d // HQ
        D = self.D
        pages, self.table, _ = _tables(B, length, 0)
        self.cache = _cache(pages, bits, D)
        self.rope = moeq4.RopeSpec(moeq4.moe_rope_phases(D, 1e6).cuda(), D)
        self.lens = torch.full((B,), length, dtype=torch.int32, device="cuda")
        self.pos = self.lens - 1                       # the new token is the context's last
        last = (self.pos // self.cache.page_size).long()
        self.slots = (self.table.gather(1, last[:, None])[:, 0] * self.cache.page_size
                      + self.pos % self.cache.page_size).int()
        self.att = torch.empty((B, HQ, D), dtype=torch.bfloat16, device="cuda")
        self.ws = moeq4.alloc_workspace(
            moeq4.moe_kv_attention_workspace_size(B, 1, HQ, HKV, D, length, 0))

    def __call__(self, qkv):
        """The attention [B, HQ * D] of the projected rows qkv [B, HQ + 2 HKV, D]."""
        q = qkv[:, :HQ]
        moeq4.moe_kv_append(self.cache, qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], self.slots, self.pos,
                            self.rope, q, q)
        moeq4.moe_kv_attention(q, self.cache, self.table, self.lens, self.length, self.att, self.ws)
        return self.att.view(self.B, -1)


def _weights(n: int, k: int) -> torch.Tensor:
    return torch.randn((n, k), device="cuda").mul_(k ** -0.5).bfloat16()


def _step(B: int, length: int, bits: int, calls: int) -> None:
    cfg = dataclasses.replace(synth.CONFIGS["t512"], T=B)
    W = moeq4.DeviceWeights.from_host(synth.gen_weights(cfg, 0))
    lay = moeq4.Layer(W, B, cfg.k, None)
    lg = torch.from_numpy(synth.gen_logits(cfg, 0, B)).cuda()
    x = torch.from_numpy(synth.gen_x(cfg, B).view(np.int16)).cuda().view(torch.bfloat16)
    attend = _Attention(cfg, B, length, bits)
    w_qkv = _weights((HQ + 2 * HKV) * attend.D, cfg.d).t().contiguous()
    w_out = _weights(cfg.d, HQ * attend.D).t().contiguous()

    def step():
        qkv = (x @ w_qkv).view(B, HQ + 2 * HKV, attend.D)
        return lay(x + attend(qkv) @ w_out, lg)

    _timed(step, calls, attend.cache)
    _clean(lay.route)


def _block(B: int, length: int, bits: int, calls: int) -> None:
    cfg = dataclasses.replace(synth.CONFIGS["t512"], T=B)
    W = moeq4.DeviceWeights.from_host(synth.gen_weights(cfg, 0))
    route = moeq4.RouteBuffers.alloc(B, cfg.E, cfg.k, moeq4.default_block_m(B, cfg.E, cfg.k))
    ws = moeq4.alloc_workspace(moeq4.moe_layer_workspace_size(B, cfg.E, cfg.k, W.d, W.f, W.f_s,
                                                              route.block_m))
    x = torch.from_numpy(synth.gen_x(cfg, B).view(np.int16)).cuda().view(torch.bfloat16)
    ones = torch.ones(cfg.d, dtype=torch.bfloat16, device="cuda")
    router = moeq4.Linear(_weights(cfg.E, cfg.d))
    score = moeq4.RouteScore(moeq4.MOE_SCORE_SIGMOID, 0.1 * torch.randn(cfg.E, device="cuda"),
                             groups=8, top_groups=4, group_best=2, factor=2.5)
    attend = _Attention(cfg, B, length, bits)
    heads, D = HQ + 2 * HKV, attend.D
    qkv, out = moeq4.Linear(_weights(heads * D, cfg.d)), moeq4.Linear(_weights(cfg.d, HQ * D))
    rows = torch.empty((B, heads, D), dtype=torch.bfloat16, device="cuda")
    h1, n1, h2, n2, y = (torch.zeros_like(x) for _ in range(5))
    lg = torch.empty((B, cfg.E), dtype=torch.float32, device="cuda")

    def block():
        # y: the experts' output of the layer before (here: of the call before)
        moeq4.moe_rms_norm(x, ones, n1, add=y, sum=h1)
        moeq4.moe_linear(n1, qkv, rows.view(B, -1))
        moeq4.moe_rms_norm(rows[:, :HQ + HKV], ones[:D], rows[:, :HQ + HKV])
        moeq4.moe_linear(attend(rows), out, h2, add=h1)
        moeq4.moe_rms_norm(h2, ones, n2)
        moeq4.moe_linear(n2, router, lg)
        moeq4.moe_layer_scored(n2, lg, W, score, route, y, ws)

    _timed(block, calls, attend.cache)
    _clean(route, qkv, out, router)


def _clean(*owners) -> None:
    if any(moeq4.moe_get_device_error(o) for o in owners):
        raise RuntimeError("device error word set")


def _linear(T: int, N: int, K: int, e4m3: int, calls: int) -> None:
    x, w, scale = torch.randn((T, K), device="cuda"), torch.randn((N, K), device="cuda"), None
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    if e4m3:
        scale = torch.full((max(T, N),), K ** -0.25, device="cuda")
    lin = moeq4.Linear(w.to(dtype), None, scale[:N].contiguous() if e4m3 else None)
    x, xs = x.to(dtype), scale[:T].contiguous() if e4m3 else None
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    _timed(lambda: moeq4.moe_linear(x, lin, out, x_scale=xs), calls, lin)


def _norm(T: int, D: int, codes: int, calls: int) -> None:
    x, add = (torch.randn((T, D), device="cuda").bfloat16() for _ in range(2))
    weight, total = torch.ones_like(x[0]), torch.empty_like(x)
    if codes:
        kw = dict(codes=torch.empty((T, D), dtype=torch.float8_e4m3fn, device="cuda"),
                  scales=torch.empty(T, device="cuda"))
    else:
        kw = dict(out=torch.empty_like(x))
    _timed(lambda: moeq4.moe_rms_norm(x, weight, add=add, sum=total, **kw), calls)


def _scored(T: int, E: int, groups: int, calls: int) -> None:
    lg = 1.5 * torch.randn((T, E), device="cuda")
    score = moeq4.RouteScore(moeq4.MOE_SCORE_SIGMOID, 0.1 * torch.randn(E, device="cuda"), groups,
                             max(1, groups // 2), 2 if groups > 1 else 1, factor=2.5)
    out = moeq4.RouteBuffers.alloc(T, E, 8)
    ws = moeq4.alloc_workspace(moeq4.moe_route_workspace_size(T, E, 8))
    _timed(lambda: moeq4.moe_route_scored(lg, score, out, ws), calls, out)


def _timed(fn, calls: int, owner=None) -> None:
    fn()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(calls - 1):
        fn()
    e1.record()
    torch.cuda.synchronize()
    us = e0.elapsed_time(e1) / max(1, calls - 1) * 1e3
    said = "" if owner is None else f"; device error word {moeq4.moe_get_device_error(owner)}"
    print(f"mean {us:.1f} us per call over {calls - 1} calls{said}")


def main(argv) -> None:
    what, nums = argv[1], [int(v) for v in argv[2:]]
    if what == "attention":
        B, nq, length, prefix, bits, D, calls = nums + [8, 128, 4][len(nums) - 4:]
        _attention(B, nq, length, prefix, bits, D, calls)
    elif what in ("step", "block"):
        B, length, bits, calls = nums + [8, 4][len(nums) - 2:]
        {"step": _step, "block": _block}[what](B, length, bits, calls)
    elif what == "linear":
        _linear(*(nums + [0, 4][len(nums) - 3:]))
    elif what == "norm":
        _norm(*(nums + [0, 4][len(nums) - 2:]))
    elif what == "scored":
        _scored(*(nums + [4][len(nums) - 3:]))
    else:
        {"layer": _layer, "router": _router}[what](nums[0], nums[1] if len(nums) > 1 else 4)


if __name__ == "__main__":
    main(sys.argv)
