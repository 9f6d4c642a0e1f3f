"""The attention-side operators of a serving step, as measured cases.

Next to the expert layer a decoder layer turns its queries and keys by their
positions, keeps keys and values in a paged, quantised cache, and attends over
that cache. Five operations, four calls:

* ``rope``    rotary positions on heads of any stride, forward or gradient
* ``append``  rotary positions, then keys and values quantised (groups of 64
              along the head, 8 or 4 bits, one bf16 scale and bias per group)
              into their cache slots; the written rows are read back
* ``read``    cache rows back as bf16
* ``attend``  attention over each request's pages: one or more query tokens per
              request (causal among themselves), lengths from zero up
* ``prefix``  the same call when all requests also share one long prefix

``own`` false computes them from elementary torch operations in fp32, ``own``
true through the framework's calls. Cache layout, shared by both: a page holds
the keys of each head, then the values of each head; one head's part is its
codes ``[page_size][D * bits / 8]`` (4-bit: code 2i of a row in the low nibble
of byte i) followed by its words ``[page_size][D / 64]``, scale in the low and
bias in the high 16 bits, both bf16. A value is ``scale * code + bias``.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 64          # elements that share a scale and a bias


# ------------------------------------------------------------------ cases

def listed():
    return [
        # rotary positions of one decoded token: fused query and key heads of one row
        dict(name="rope_token", op="rope", T=1, Hq=16, Hkv=2, D=128, rot=128, interleaved=False,
             base=10000.0, factor=1.0, mscale=1.0, top=32768, backward=False, dtype="bf16"),
        # gradient of the rotation over an odd number of tokens, fp32, half of each head,
        # positions stretched for a long context
        dict(name="rope_gradient", op="rope", T=2047, Hq=32, Hkv=8, D=128, rot=64,
             interleaved=True, base=1000000.0, factor=4.0, mscale=1.1386, top=131072,
             backward=True, dtype="f32"),
        # one decode step of 64 requests
        dict(name="append_step", op="append", T=64, Hq=16, Hkv=2, D=128, rot=128,
             interleaved=False, base=10000.0, factor=1.0, mscale=1.0, top=32768, bits=8,
             page_size=16),
        # one 4096-token chunk of a long prompt
        dict(name="append_chunk", op="append", T=4096, Hq=32, Hkv=8, D=128, rot=64,
             interleaved=False, base=1000000.0, factor=2.0, mscale=1.07, top=131072, bits=4,
             page_size=64),
        # a short request's rows moved out of the cache
        dict(name="read_request", op="read", n=333, Hkv=2, D=256, bits=8, page_size=32),
        # a whole 32K context moved out of the cache
        dict(name="read_context", op="read", n=32768, Hkv=8, D=128, bits=4, page_size=64),
        # one request, a few hundred tokens: latency
        dict(name="attend_token", op="attend", B=1, nq=1, Hq=16, Hkv=2, D=128, bits=8,
             page_size=16, longest=777, shortest=777, prefix=0),
        # one request with a 128K context: the length is the only axis to split
        dict(name="attend_long", op="attend", B=1, nq=1, Hq=32, Hkv=8, D=128, bits=8,
             page_size=64, longest=131071, shortest=131071, prefix=0),
        # a batch of decoding requests of very different lengths, empty ones among them
        dict(name="attend_batch", op="attend", B=64, nq=1, Hq=32, Hkv=8, D=128, bits=4,
             page_size=64, longest=8192, shortest=0, prefix=0),
        # the last 4096-token chunk of a 32K prompt over its quantised cache
        dict(name="attend_chunk", op="attend", B=1, nq=4096, Hq=16, Hkv=2, D=128, bits=8,
             page_size=128, longest=32768, shortest=32768, prefix=0),
        # 64 requests behind one system prompt
        dict(name="prefix_batch", op="prefix", B=64, nq=1, Hq=16, Hkv=2, D=256, bits=4,
             page_size=48, longest=600, shortest=1, prefix=16000),
        # drafts of four tokens checked for 128 requests behind a shared document
        dict(name="prefix_drafts", op="prefix", B=128, nq=4, Hq=16, Hkv=2, D=128, bits=8,
             page_size=64, longest=1024, shortest=0, prefix=65536),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(("rope", "append", "read", "attend", "attend", "prefix", "prefix"))
    Hq, Hkv = rng.choice(((16, 2), (32, 8), (8, 8), (16, 1), (24, 4), (20, 4), (6, 2), (64, 8)))
    D = rng.choice((64, 128, 256))
    case = dict(op=op, Hq=Hq, Hkv=Hkv, D=D)
    if op in ("rope", "append"):
        factor = rng.choice((1.0, 1.0, 2.0, 4.0, 8.0))
        case.update(T=_log(rng, 1, 8192), rot=rng.choice((D, D, D // 2, D // 4, D // 2 + 8)),
                    interleaved=rng.random() < 0.5, base=rng.choice((10000.0, 500000.0, 1e6)),
                    factor=factor, mscale=round(1.0 + 0.1 * math.log(factor), 4),
                    top=rng.choice((2048, 32768, 131072, 1000000)))
        if op == "rope":
            case.update(backward=rng.random() < 0.5, dtype=rng.choice(("bf16", "f16", "f32")))
            return case
    case.update(bits=rng.choice((8, 4)), page_size=rng.choice((16, 32, 48, 64, 128, 256)))
    if op == "read":
        case.update(n=_log(rng, 1, 131072 // max(1, Hkv * D // 512)))
    elif op == "attend":
        kind = rng.choice(("step", "step", "drafts", "chunk"))
        nq = {"step": 1, "drafts": rng.randint(2, 8), "chunk": _log(rng, 9, 2048)}[kind]
        B = _log(rng, 1, 256 if kind != "chunk" else 4)
        most = min(131072, 256 * 1024 * 1024 // (B * Hkv * D),
                   1024 * 1024 * 1024 // (B * nq * Hq))
        longest = _log(rng, max(1, nq), max(nq, most))
        case.update(B=B, nq=nq, longest=longest, prefix=0,
                    shortest=rng.choice((0, longest // 3, longest)))
    elif op == "prefix":
        nq = rng.choice((1, 1, 1, rng.randint(2, 6)))
        B = _log(rng, 2, 256)
        longest = _log(rng, 1, max(1, min(2048, 128 * 1024 * 1024 // (B * Hkv * D))))
        most = min(131072, 1024 * 1024 * 1024 // (B * nq * Hq))
        case.update(B=B, nq=nq, longest=longest, shortest=rng.choice((0, longest)),
                    prefix=_log(rng, 64, max(64, most)))
    return case


def _lens(case):
    """Context length of each request: between shortest and longest, both present."""
    B, lo, hi = case["B"], case["shortest"], case["longest"]
    r = random.Random(B * 1000003 + hi)
    lens = [r.randint(lo, hi) for _ in range(B)]
    lens[0] = hi
    if B > 2:
        lens[B // 2] = lo
    return lens


def work(case):
    op, D = case["op"], case["D"]
    if op == "rope":
        es = 4 if case["dtype"] == "f32" else 2
        H, T = case["Hq"] + case["Hkv"], case["T"]
        return dict(bytes=2 * T * H * D * es + 4 * T + 4 * case["rot"],
                    flops=3 * T * H * case["rot"])
    row = 2 * case["Hkv"] * (D * case["bits"] // 8 + D // GROUP * 4)   # one token's keys and values
    values = 2 * case["Hkv"] * D
    if op == "append":
        T, Hq = case["T"], case["Hq"]
        return dict(bytes=T * (2 * values + 4 * Hq * D + row + 8 + row + 2 * values + 4)
                    + 4 * case["rot"],
                    flops=T * (3 * (Hq + case["Hkv"]) * case["rot"] + 6 * values))
    if op == "read":
        return dict(bytes=case["n"] * (row + 2 * values + 4), flops=2 * case["n"] * values)
    lens, nq, P = _lens(case), case["nq"], case["page_size"]
    seen = sum(max(0, n - nq + 1 + i) for n in lens for i in range(nq))
    pages = sum(-(-n // P) for n in lens) + -(-case["prefix"] // P)
    return dict(bytes=(sum(lens) + case["prefix"]) * row + 4 * pages + 4 * case["B"]
                + 4 * case["B"] * nq * case["Hq"] * D,
                flops=4 * D * case["Hq"] * (seen + case["B"] * nq * case["prefix"]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _phases(case):
    """Turns per position of each pair, as 64-bit fractions of a turn; positions
    divided by `factor` for contexts beyond the trained length."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64)
    turns = case["base"] ** (-2.0 * i / case["rot"]) / (2.0 * math.pi * case["factor"])
    return (turns * 2.0 ** 64).to(torch.int64).cuda()


def _positions(case, T, g):
    """Tokens of several requests: runs of consecutive positions."""
    start = torch.randint(0, case["top"], (T // 128 + 1,), generator=g, device="cuda")
    i = torch.arange(T, device="cuda")
    return ((start[i // 128] + i % 128) % case["top"]).to(torch.int32)


def _head_bytes(case):
    P, D = case["page_size"], case["D"]
    return P * D * case["bits"] // 8, P * (D // GROUP) * 4


def _empty_cache(case, pages):
    """Pages no one has written: their bytes are whatever memory held (here 0xFF,
    which reads as NaN where a scale or bias would be)."""
    cb, mb = _head_bytes(case)
    return torch.full((pages, 2, case["Hkv"], cb + mb), 255, dtype=torch.uint8, device="cuda")


def _filled_cache(case, pages, g):
    """Pages of quantised normal values; keys have a few wide groups."""
    data = _empty_cache(case, pages)
    cb, mb = _head_bytes(case)
    Hkv, P, nb = case["Hkv"], case["page_size"], case["D"] // GROUP
    step = max(1, (1 << 27) // (2 * Hkv * cb))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        z = torch.empty((n, 2, Hkv, cb * (8 // case["bits"])), dtype=torch.float16, device="cuda")
        z.normal_(generator=g)
        if case["bits"] == 8:
            data[p:p + n, ..., :cb] = z.mul_(46.0).add_(127.5).round_().clamp_(0, 255).to(torch.uint8)
        else:
            q = z.mul_(4.0).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
            data[p:p + n, ..., :cb] = q[..., ::2] | (q[..., 1::2] << 4)
        levels = 2 ** case["bits"] - 1
        span = torch.empty((n, 2, Hkv, P, nb), device="cuda").uniform_(4.0, 6.0, generator=g)
        span[:, 0, :, :, 0] *= 1.5
        sb = torch.stack((span / levels, span * -0.5), -1).to(torch.bfloat16)
        data[p:p + n, ..., cb:] = sb.view(torch.uint8).reshape(n, 2, Hkv, mb)
    return data


def _stale(data, case, pages, first):
    """Slots from `first` on in each of `pages` were never written: NaN words."""
    cb, mb = _head_bytes(case)
    P = case["page_size"]
    words = data[..., cb:].unflatten(-1, (P, mb // P))
    off = torch.arange(P, device="cuda")[None] >= first[:, None]
    at = torch.nonzero(off)
    words[pages[at[:, 0]], :, :, at[:, 1]] = 255


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    D = case["D"]
    if case["op"] == "rope":
        dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[case["dtype"]]
        T, H = case["T"], case["Hq"] + case["Hkv"]
        qkv = torch.randn((T, H + case["Hkv"], D), generator=g, device="cuda").to(dt)
        s.update(x=qkv[:, :H], out=torch.empty((T, H, D), dtype=dt, device="cuda"),
                 pos=_positions(case, T, g), phase=_phases(case))
        return s
    Hkv, P = case["Hkv"], case["page_size"]
    if case["op"] == "append":
        T, Hq = case["T"], case["Hq"]
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        pages = -(-T // P) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(T, device="cuda")
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:],
                 slots=(order[i // P] * P + i % P).to(torch.int32), pos=_positions(case, T, g),
                 phase=_phases(case), data=_empty_cache(case, pages),
                 q_out=torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda"),
                 k_out=torch.empty((T, Hkv, D), dtype=torch.bfloat16, device="cuda"),
                 v_out=torch.empty((T, Hkv, D), dtype=torch.bfloat16, device="cuda"))
        return s
    if case["op"] == "read":
        n = case["n"]
        pages = -(-n // P) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(n, device="cuda")
        s.update(data=_filled_cache(case, pages, g),
                 slots=(order[i // P] * P + i % P).to(torch.int32),
                 k_out=torch.empty((n, Hkv, D), dtype=torch.bfloat16, device="cuda"),
                 v_out=torch.empty((n, Hkv, D), dtype=torch.bfloat16, device="cuda"))
        return s
    lens, B, nq, Hq = _lens(case), case["B"], case["nq"], case["Hq"]
    per, pre = max(1, -(-case["longest"] // P)), -(-case["prefix"] // P)
    n = torch.tensor(lens, device="cuda")
    used = (n + P - 1) // P
    base = torch.cumsum(used, 0) - used
    total = sum(-(-x // P) for x in lens) + pre
    order = torch.randperm(total + 3, generator=g, device="cuda")
    j = torch.arange(per, device="cuda")[None]
    # entries past a request's last page were never set
    table = torch.where(j < used[:, None], order[(base[:, None] + j).clamp(max=total)], -1)
    data = _filled_cache(case, total + 3, g)
    some = torch.nonzero(n % P)[:, 0]
    _stale(data, case, order[base[some] + used[some] - 1], n[some] % P)
    prefix_table = order[total - pre:total]
    if case["prefix"] % P:
        _stale(data, case, prefix_table[-1:], torch.tensor([case["prefix"] % P], device="cuda"))
    qkv = torch.randn((B * nq, Hq + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    s.update(q=qkv[:, :Hq], data=data, table=table.to(torch.int32).contiguous(),
             lens=n.to(torch.int32), prefix_table=prefix_table.to(torch.int32),
             out=torch.empty((B * nq, Hq, D), dtype=torch.bfloat16, device="cuda"))
    return s


# ------------------------------------------------------------- plain form

def _turned(x, pos, phase, case, sign):
    """fp32 x [T][H][D] turned by pos * phase (mod one turn)."""
    angle = ((pos.long()[:, None] * phase[None]) >> 32).float() * (math.pi / 2 ** 31)
    c = (angle.cos() * case["mscale"])[:, None]
    s = (angle.sin() * case["mscale"] * sign)[:, None]
    rot = case["rot"]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _quantised(x, bits):
    """bf16 x [T][H][D] as the values its codes stand for, fp32."""
    v = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    levels = 2 ** bits - 1
    scale = ((hi * 0.5 - lo * 0.5) / (0.5 * levels)).bfloat16().float()
    per = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
    code = ((v - lo) * per).round().clamp(0, levels)
    return (scale * code + lo).flatten(-2)


def _values(data, case):
    """Pages [..., Hkv, head bytes] as fp32 values [..., Hkv, page_size, D]."""
    cb, mb = _head_bytes(case)
    P, D = case["page_size"], case["D"]
    c = data[..., :cb]
    if case["bits"] == 4:
        c = torch.stack((c & 15, c >> 4), -1).flatten(-2)
    sb = data[..., cb:].contiguous().view(torch.bfloat16).float()
    sb = sb.unflatten(-1, (P, D // GROUP, 2))
    c = c.float().unflatten(-1, (P, D // GROUP, GROUP))
    return (c * sb[..., :1] + sb[..., 1:]).flatten(-2)


def _attended(s):
    case = s["case"]
    B, nq, Hq, Hkv, D = (case[x] for x in ("B", "nq", "Hq", "Hkv", "D"))
    q = s["q"].float() * (1.0 / math.sqrt(D))
    q = q.view(B, nq, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    kv = _values(s["data"][s["table"].long().clamp(min=0)], case)     # [B][pages][2][Hkv][P][D]
    kv = kv.permute(2, 0, 3, 1, 4, 5).flatten(3, 4)                   # [2][B][Hkv][L][D]
    at = torch.arange(kv.shape[3], device="cuda")
    n = s["lens"].long()
    own_kv = (at[None] < n[:, None])[:, None, :, None]
    k, v = kv[0], torch.where(own_kv, kv[1], 0.0)
    seen = n[:, None] - nq + 1 + torch.arange(nq, device="cuda")[None]
    ok = at[None, None] < seen[..., None]                             # [B][nq][L]
    ok = ok[:, None, :, None].expand(B, 1, nq, Hq // Hkv, -1).reshape(B, 1, nq * Hq // Hkv, -1)
    logits = (q @ k.transpose(-1, -2)).masked_fill(~ok, -math.inf)
    top = logits.amax(-1, keepdim=True)
    if case["prefix"]:
        pk, pv = _values(s["data"][s["prefix_table"].long()], case).permute(1, 2, 0, 3, 4) \
            .flatten(2, 3)[:, :, :case["prefix"]]                     # [Hkv][prefix][D]
        rows = q.transpose(0, 1).reshape(Hkv, -1, D)
        shared = rows @ pk.transpose(-1, -2)
        top = torch.maximum(top, shared.amax(-1).view(Hkv, B, -1, 1).transpose(0, 1))
    top = torch.where(top > -math.inf, top, 0.0)
    p = (logits - top).exp()
    total, y = p.sum(-1, keepdim=True), p @ v
    if case["prefix"]:
        p = (shared - top.transpose(0, 1).reshape(Hkv, -1, 1)).exp()
        total = total + p.sum(-1).view(Hkv, B, -1, 1).transpose(0, 1)
        y = y + (p @ pv).view(Hkv, B, -1, D).transpose(0, 1)
    y = torch.where(total > 0, y / total, 0.0)
    y = y.view(B, Hkv, nq, Hq // Hkv, D).transpose(1, 2)
    return y.reshape(B * nq, Hq, D).bfloat16()


def _plain(s):
    case = s["case"]
    if case["op"] == "rope":
        sign = -1.0 if case["backward"] else 1.0
        return _turned(s["x"].float(), s["pos"], s["phase"], case, sign).to(s["x"].dtype)
    if case["op"] == "append":
        q = _turned(s["q"].float(), s["pos"], s["phase"], case, 1.0).bfloat16()
        k = _turned(s["k"].float(), s["pos"], s["phase"], case, 1.0).bfloat16()
        return (q, _quantised(k, case["bits"]).bfloat16(),
                _quantised(s["v"], case["bits"]).bfloat16())
    if case["op"] == "read":
        P = case["page_size"]
        slots = s["slots"].long()
        rows = _values(s["data"][slots[::P] // P], case)              # whole pages, in order
        rows = rows.permute(1, 0, 3, 2, 4).flatten(1, 2)[:, :case["n"]].bfloat16()
        return rows[0], rows[1]
    return _attended(s)


# -------------------------------------------------------- framework's calls

def _handles(s):
    """The structures a program keeps beside its tensors."""
    from routing_q4_grouped_gb300 import moeq4
    case, h = s["case"], {"moeq4": moeq4}
    if "phase" in s:
        h["rope"] = moeq4.RopeSpec(s["phase"], case["rot"], case["interleaved"], case["mscale"])
    if "data" in s:
        h["cache"] = moeq4.KVCache(s["data"], case["page_size"], case["Hkv"], case["D"],
                                   case["bits"])
    if "lens" in s:
        h["ws"] = moeq4.alloc_workspace(moeq4.moe_kv_attention_workspace_size(
            case["B"], case["nq"], case["Hq"], case["Hkv"], case["D"], case["longest"],
            case["prefix"]))
    return h


def _calls(s):
    case = s["case"]
    h = s.get("handles") or s.setdefault("handles", _handles(s))
    moeq4 = h["moeq4"]
    if case["op"] == "rope":
        moeq4.moe_rope(s["x"], s["out"], s["pos"], h["rope"], backward=case["backward"])
        return s["out"]
    if case["op"] == "append":
        moeq4.moe_kv_append(h["cache"], s["k"], s["v"], s["slots"], s["pos"], h["rope"], s["q"],
                            s["q_out"])
        moeq4.moe_kv_read(h["cache"], s["slots"], s["k_out"], s["v_out"])
        return s["q_out"], s["k_out"], s["v_out"]
    if case["op"] == "read":
        moeq4.moe_kv_read(h["cache"], s["slots"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    shared = dict(prefix_table=s["prefix_table"], prefix_len=case["prefix"]) if case["prefix"] else {}
    moeq4.moe_kv_attention(s["q"], h["cache"], s["table"], s["lens"], case["longest"], s["out"],
                           h["ws"], nq=case["nq"], **shared)
    return s["out"]


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------- the definition, 64 bits

def _turn64(x, s):
    """x [T][H][D] float64 turned by its positions."""
    case = s["case"]
    pos = s["pos"].cpu().numpy().astype(np.int64).astype(np.uint64)
    phase = s["phase"].cpu().numpy().astype(np.uint64)
    with np.errstate(over="ignore"):
        frac = (pos[:, None] * phase[None]).astype(np.float64) / 2.0 ** 64
    a = torch.from_numpy(2.0 * np.pi * frac).cuda()[:, None]
    if case.get("backward"):
        a = -a
    half = case["rot"] // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    y = x.clone()
    m = case["mscale"]
    y[..., first] = m * (x[..., first] * torch.cos(a) - x[..., second] * torch.sin(a))
    y[..., second] = m * (x[..., second] * torch.cos(a) + x[..., first] * torch.sin(a))
    return y


def _codes64(x, bits):
    """Values of x [T][H][D] after quantisation with a bf16 scale and bias per group."""
    T, H, D = x.shape
    g = x.double().reshape(T, H, D // GROUP, GROUP)
    low = g.min(-1).values
    scale = ((g.max(-1).values - low) / (2 ** bits - 1)).to(torch.bfloat16).double()
    safe = torch.where(scale > 0, scale, 1.0)
    code = torch.round((g - low[..., None]) / safe[..., None]).clamp(0, 2 ** bits - 1)
    return (low[..., None] + scale[..., None] * code).reshape(T, H, D)


def _rows64(s, pages, count):
    """The first `count` tokens of the listed pages: keys, values [Hkv][count][D] float64."""
    case = s["case"]
    P, D, bits = case["page_size"], case["D"], case["bits"]
    raw = s["data"][pages.long()]                                     # [n][2][Hkv][bytes]
    row = D * bits // 8
    codes = raw[..., :P * row].reshape(*raw.shape[:3], P, row)
    if bits == 4:
        wide = torch.empty((*codes.shape[:-1], D), dtype=torch.uint8, device="cuda")
        wide[..., 0::2] = codes % 16
        wide[..., 1::2] = codes // 16
        codes = wide
    words = raw[..., P * row:].contiguous().view(torch.bfloat16)
    words = words.reshape(*raw.shape[:3], P, D // GROUP, 2).double()
    scale = words[..., 0].repeat_interleave(GROUP, -1)
    bias = words[..., 1].repeat_interleave(GROUP, -1)
    val = torch.addcmul(bias, scale, codes.double())                  # [n][2][Hkv][P][D]
    val = val.permute(1, 2, 0, 3, 4).reshape(2, case["Hkv"], -1, D)[:, :, :count]
    return val[0], val[1]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turn64(s["x"].double(), s)
    if case["op"] == "append":
        k = _turn64(s["k"].double(), s).to(torch.bfloat16)
        return (_turn64(s["q"].double(), s), _codes64(k, case["bits"]),
                _codes64(s["v"], case["bits"]))
    if case["op"] == "read":
        first = s["slots"][::case["page_size"]] // case["page_size"]
        k, v = _rows64(s, first, case["n"])
        return k.transpose(0, 1), v.transpose(0, 1)
    B, nq, Hq, Hkv, D, P = (case[x] for x in ("B", "nq", "Hq", "Hkv", "D", "page_size"))
    G = Hq // Hkv
    y = torch.zeros((B, nq, Hq, D), dtype=torch.float64, device="cuda")
    q = s["q"].double().reshape(B, nq, Hq, D)
    shared = _rows64(s, s["prefix_table"], case["prefix"])
    for b, n in enumerate(_lens(case)):
        own_rows = _rows64(s, s["table"][b, :max(1, -(-n // P))].clamp(min=0), n)
        for h in range(Hkv):
            k = torch.cat((shared[0][h], own_rows[0][h]))
            v = torch.cat((shared[1][h], own_rows[1][h]))
            limit = case["prefix"] + n - nq + 1 + torch.arange(nq, device="cuda")
            limit = torch.maximum(limit, torch.full_like(limit, case["prefix"]))
            at = torch.arange(k.shape[0], device="cuda")
            for g in range(h * G, h * G + G):
                z = (q[b, :, g] @ k.T) / math.sqrt(D)
                z.masked_fill_(at[None] >= limit[:, None], -math.inf)
                w = torch.softmax(z, -1)
                y[b, :, g] = torch.where((limit > 0)[:, None], w, 0.0) @ v
    return y.reshape(B * nq, Hq, D)
