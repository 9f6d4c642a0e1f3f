"""The calls of a decoder layer in a row, as a program makes them: residual and norm, the fused
projection, per-head norm, append, attention, output projection with the residual, norm, router
logits, routing by scores, experts; eagerly and captured, with 16-bit and 8-bit projections.

Each call is tested on its own elsewhere; here the chain is checked against the same chain in
float64, call by call from the tensors that the library produced (so that a rounding at one step
does not count at the next), with each call's own bound.
"""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_helpers import assert_y_close, bits
from oracle import scored
from routing_q4_grouped_gb300 import moeq4, synth

pytestmark = pytest.mark.gpu

B, D, HQ, HKV, PAGE = 12, 64, 4, 2, 16
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


class Block:
    def __init__(self, codes: bool):
        cfg = synth.CONFIGS["tiny"]
        self.cfg, self.codes = cfg, codes
        g = torch.Generator(device="cuda").manual_seed(1)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")      # noqa: E731
        d, H = cfg.d, HQ + 2 * HKV
        self.Wh = synth.gen_weights(cfg)
        self.W = moeq4.DeviceWeights.from_host(self.Wh)
        w = rnd(H * D, d) * d ** -0.5
        self.qkv_bias = 0.1 * rnd(H * D)
        if codes:
            ws = w.abs().amax(-1) / 448
            self.w_qkv = (w / ws[:, None]).to(E4M3)
            self.qkv = moeq4.Linear(self.w_qkv, self.qkv_bias, ws)
        else:
            self.w_qkv = w.to(BF16)
            self.qkv = moeq4.Linear(self.w_qkv, self.qkv_bias)
        self.w_out = (rnd(d, HQ * D) * (HQ * D) ** -0.5).to(BF16)
        self.w_router = (rnd(cfg.E, d) * d ** -0.5).to(BF16)
        self.out, self.router = moeq4.Linear(self.w_out), moeq4.Linear(self.w_router)
        self.n1, self.n2 = (1 + 0.1 * rnd(d)).to(BF16), (1 + 0.1 * rnd(d)).to(BF16)
        self.nq = (1 + 0.1 * rnd(D)).to(BF16)
        self.bias = 0.05 * rnd(cfg.E)
        self.spec = moeq4.RouteScore(moeq4.MOE_SCORE_SIGMOID, self.bias, 4, 2, 1, True, 1.5)
        self.h = rnd(B, d).to(BF16)
        self.delta = rnd(B, d).to(BF16)
        E = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        self.h1, self.x1, self.h2, self.x2, self.y = (E(B, d) for _ in range(5))
        self.c1, self.s1 = E(B, d, dt=E4M3), E(B, dt=torch.float32)
        self.t_qkv, self.att = E(B, H * D), E(B, HQ, D)
        self.qk = E(B, HQ + HKV, D)
        self.logits = E(B, cfg.E, dt=torch.float32)
        self.cache = moeq4.KVCache.alloc(B * 4, PAGE, HKV, D, 8)
        self.table = torch.randperm(B * 4, generator=g, device="cuda").int().view(B, 4)
        self.lens = torch.randint(20, 64, (B,), generator=g, device="cuda", dtype=torch.int32)
        old = rnd(B * 4 * PAGE, 2 * HKV, D).to(BF16)
        moeq4.moe_kv_append(self.cache, old[:, :HKV], old[:, HKV:],
                            torch.arange(B * 4 * PAGE, dtype=torch.int32, device="cuda"))
        self.pos = self.lens - 1
        self.slots = (self.table.gather(1, (self.pos // PAGE).long()[:, None])[:, 0] * PAGE
                      + self.pos % PAGE).int()
        self.rope = moeq4.RopeSpec(moeq4.moe_rope_phases(D, 10000.0).cuda(), D)
        self.r = moeq4.RouteBuffers.alloc(B, cfg.E, cfg.k)
        self.ws = moeq4.alloc_workspace(moeq4.moe_layer_workspace_size(
            B, cfg.E, cfg.k, cfg.d, cfg.f, cfg.f_s, 128))
        self.ws_att = moeq4.alloc_workspace(moeq4.moe_kv_attention_workspace_size(
            B, 1, HQ, HKV, D, 64))

    def run(self):
        if self.codes:
            moeq4.moe_rms_norm(self.h, self.n1, add=self.delta, sum=self.h1, codes=self.c1,
                               scales=self.s1)
            moeq4.moe_linear(self.c1, self.qkv, self.t_qkv, x_scale=self.s1)
        else:
            moeq4.moe_rms_norm(self.h, self.n1, self.x1, add=self.delta, sum=self.h1)
            moeq4.moe_linear(self.x1, self.qkv, self.t_qkv)
        qkv = self.t_qkv.view(B, HQ + 2 * HKV, D)
        moeq4.moe_rms_norm(qkv[:, :HQ + HKV], self.nq, self.qk)
        q = self.qk[:, :HQ]
        moeq4.moe_kv_append(self.cache, self.qk[:, HQ:], qkv[:, HQ + HKV:], self.slots, self.pos,
                            self.rope, q, q)
        moeq4.moe_kv_attention(q, self.cache, self.table, self.lens, 64, self.att, self.ws_att)
        moeq4.moe_linear(self.att.view(B, -1), self.out, self.h2, add=self.h1)
        moeq4.moe_rms_norm(self.h2, self.n2, self.x2)
        moeq4.moe_linear(self.x2, self.router, self.logits)
        moeq4.moe_layer_scored(self.x2, self.logits, self.W, self.spec, self.r, self.y, self.ws)

    def results(self):
        return [t.clone() for t in (self.h1, self.t_qkv, self.qk, self.att, self.h2, self.x2,
                                    self.logits, self.r.ids, self.r.w, self.y)]


def _norm64(x, w):
    x = x.double()
    return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()


def _close(got, want, more=0.0):
    # one rounding to bf16, the arithmetic of the call (far below it), and `more`
    bound = want.abs() * (2.0 ** -8 + 2.0 ** -12) + more + 2.0 ** -14
    assert ((got.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("codes", [False, True])
def test_layer_call_by_call(codes):
    b = Block(codes)
    b.run()
    torch.cuda.synchronize()
    for lin in (b.qkv, b.out, b.router):
        assert moeq4.moe_get_device_error(lin) == 0
    assert moeq4.moe_get_device_error(b.r) == 0 and moeq4.moe_get_device_error(b.cache) == 0
    h1 = b.h.double() + b.delta.double()
    _close(b.h1, h1)
    if codes:
        x1 = b.c1.double() * b.s1.double()[:, None]
        w = b.w_qkv.double() * b.qkv.scale.double()[:, None]
        y = _norm64(h1, b.n1)
        # a code is off by 2^-4 of its value, or by half the least step
        assert ((x1 - y).abs() <= y.abs() * 2.0 ** -4 * 1.001 + b.s1.double()[:, None] * 2.0 ** -9).all()
    else:
        _close(b.x1, _norm64(h1, b.n1))
        x1, w = b.x1.double(), b.w_qkv.double()
    _close(b.t_qkv, x1 @ w.t() + b.qkv_bias.double())
    _close(b.h2, b.att.view(B, -1).double() @ b.w_out.double().t() + b.h1.double())
    _close(b.x2, _norm64(b.h2, b.n2))
    lg = b.x2.double() @ b.w_router.double().t()
    size = b.x2.double().abs() @ b.w_router.double().abs().t()
    assert ((b.logits.double() - lg).abs() <= size * 40 * 2.0 ** -23).all()
    r = scored.route_scored(b.logits.cpu().numpy(), b.cfg.k, sigmoid=True,
                            bias=b.bias.cpu().numpy(), groups=4, top_groups=2, factor=1.5)
    assert np.array_equal(b.r.ids.cpu().numpy(), r.ids)
    assert np.allclose(b.r.w.cpu().numpy(), r.w, rtol=2.0 ** -18, atol=0)
    r.w = r.w.astype(np.float32)
    assert_y_close(bits(b.y), O.expert_ffn(bits(b.x2), b.Wh, r))


@pytest.mark.parametrize("codes", [False, True])
def test_layer_captured(codes):
    b = Block(codes)
    b.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    for _ in range(3):
        b.h.normal_()
        b.run()
        eager = b.results()
        b.y.zero_()
        g.replay()
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(eager, b.results())):
            # the experts' rows are combined by atomic additions, in any order
            assert torch.equal(x, y) if i < 9 else torch.allclose(x.float(), y.float(), rtol=0.02, atol=0.02), i
