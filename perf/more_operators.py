"""Operators that join the attention side and the expert layer, as measured cases.

Between the attention over its cache and the grouped experts a decoder layer
adds residuals and normalises, projects, and chooses experts:

* ``norm``    x + add, its root-mean-square norm with a weight, per hidden row or
              per head of a fused row; the result in the input's type, or in 8
              bits (e4m3) with one fp32 scale per row
* ``linear``  act(x w^T + bias) + add; 16-bit operands, or e4m3 operands with one
              scale per token and per output feature; 16- or 32-bit results
* ``route``   softmax or sigmoid scores, a bias that takes part in the choice
              only, groups of experts, top-k, weights; then the histogram,
              permutation and block map that the grouped experts read

``own`` false computes them from elementary torch operations, ``own`` true
through the framework's calls.
"""
import math

import torch

own = False

TOP = 448.0                       # largest e4m3 value
LEAST = 2.0 ** -126               # smallest scale of a row of codes
BLOCK_M = 128                     # rows per entry of the block map
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
      "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token's hidden row: residual addition and norm, latency
        dict(name="norm_token", op="norm", T=1, H=1, D=2048, gap=0, dtype="bf16", add=True,
             weight=True, offset=0.0, eps=1e-6, codes=False),
        # query heads of an odd number of tokens, inside fused query/key/value rows of 20 heads
        dict(name="norm_heads", op="norm", T=2047, H=16, D=128, gap=4, dtype="f16", add=False,
             weight=True, offset=1.0, eps=1e-6, codes=False),
        # a prompt chunk's hidden rows between attention and experts
        dict(name="norm_chunk", op="norm", T=4096, H=1, D=2048, gap=0, dtype="bf16", add=True,
             weight=True, offset=0.0, eps=1e-6, codes=False),
        # long rows normalised into the 8-bit input of the next projection
        dict(name="norm_codes", op="norm", T=8191, H=1, D=5120, gap=0, dtype="bf16", add=True,
             weight=True, offset=0.0, eps=1e-5, codes=True),
        # one decoded token: sigmoid scores, balance bias, 4 of 8 groups, 8 of 256 experts
        dict(name="route_token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, best=2, renorm=True, factor=2.5),
        # a batch of decoding requests: softmax scores kept as they are
        dict(name="route_step", op="route", T=509, E=128, k=6, score="softmax", bias=False,
             groups=1, top_groups=1, best=1, renorm=False, factor=1.0),
        # a long prompt chunk through the grouped choice
        dict(name="route_chunk", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, best=2, renorm=True, factor=2.5),
        # the fused query/key/value projection of one token: the weights are read once
        dict(name="linear_token", op="linear", T=1, K=2048, N=2560, gap=0, dtype="bf16",
             out="bf16", bias=True, act="none", add=False),
        # the output projection of a decode batch, added to the residual
        dict(name="linear_step", op="linear", T=64, K=2048, N=2048, gap=0, dtype="bf16",
             out="bf16", bias=False, act="none", add=True),
        # router logits of an odd number of tokens
        dict(name="linear_router", op="linear", T=2047, K=2048, N=256, gap=0, dtype="bf16",
             out="f32", bias=False, act="none", add=False),
        # a prompt chunk through a wide projection with bias and activation
        dict(name="linear_chunk", op="linear", T=4096, K=2048, N=8192, gap=0, dtype="bf16",
             out="bf16", bias=True, act="gelu", add=False),
        # 8-bit activations and weights, the largest product
        dict(name="linear_codes", op="linear", T=8192, K=8192, N=8192, gap=0, dtype="e4m3",
             out="bf16", bias=False, act="none", add=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(("norm", "linear", "linear", "route"))
    if op == "norm":
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        H = rng.choice((1, 1, 1, 2, 8, 16, 20, 40))
        D = _log(rng, 1, 16384) if H == 1 else rng.choice((64, 80, 96, 128, 192, 256))
        T = _log(rng, 1, max(1, min(65536, (1 << 26) // (H * D))))
        return dict(op=op, T=T, H=H, D=D, gap=rng.choice((0, 0, 1, 4)), dtype=dtype,
                    add=rng.random() < 0.5, weight=rng.random() < 0.8,
                    offset=rng.choice((0.0, 0.0, 1.0)), eps=rng.choice((1e-5, 1e-6)),
                    codes=rng.random() < 0.4)
    if op == "route":
        E = rng.choice((8, 16, 60, 64, 72, 128, 160, 256, 256, 384, 512, 1024))
        kinds = [(g, t) for g, t in ((1, 1), (4, 2), (8, 4), (8, 3), (12, 5)) if E % g == 0
                 and E // g >= 2]
        groups, top = rng.choice(kinds)
        k = rng.randint(1, min(32 if E > 256 else 10, top * (E // groups)))
        return dict(op=op, T=_log(rng, 1, (1 << 22) // E), E=E, k=k,
                    score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.6,
                    groups=groups, top_groups=top, best=rng.choice((1, 2)),
                    renorm=rng.random() < 0.6, factor=rng.choice((1.0, 2.5)))
    dtype = rng.choice(("bf16", "bf16", "f16", "e4m3", "e4m3"))
    K = 16 * _log(rng, 1, 512)
    N = rng.choice((_log(rng, 1, 16384), 128 * _log(rng, 1, 128)))
    most = max(1, min(16384, (1 << 38) // (K * N)))
    T = rng.choice((_log(rng, 1, most), _log(rng, 1, min(most, 256))))
    out = rng.choice(("f32", "same", "same", "same"))
    return dict(op=op, T=T, K=K, N=N, gap=rng.choice((0, 0, 16, 64)), dtype=dtype,
                out={"same": "bf16" if dtype == "e4m3" else dtype}.get(out, out),
                bias=rng.random() < 0.5, act=rng.choice(("none", "none", "relu", "silu", "gelu",
                                                         "gelu_tanh")),
                add=rng.random() < 0.4)


def _most_tiles(case):
    rows = case["T"] * case["k"]
    return rows // BLOCK_M + min(case["E"], rows)


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        es, n = (4 if case["dtype"] == "f32" else 2), T * case["H"] * case["D"]
        per = es * (1 + 2 * case["add"]) + (1 if case["codes"] else es)
        return dict(bytes=n * per + (4 * T * case["H"] if case["codes"] else 0)
                    + (es * case["D"] if case["weight"] else 0),
                    flops=n * (5 + case["add"] + 2 * case["codes"]))
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        tiles = T * k // BLOCK_M + min(E, T * k) // 2 + 1
        return dict(bytes=4 * T * E + (4 * E if case["bias"] else 0) + 16 * T * k + 8 * E
                    + 12 * tiles, flops=T * E * 8)
    K, N = case["K"], case["N"]
    es = 1 if case["dtype"] == "e4m3" else 2
    os = 4 if case["out"] == "f32" else 2
    return dict(bytes=es * K * (T + N) + os * T * N * (1 + case["add"]) + 4 * N * case["bias"]
                + (4 * (T + N) if es == 1 else 0), flops=2 * T * N * K)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _coded(x):
    """fp32 rows as e4m3 codes and one scale per row."""
    scale = (x.abs().amax(-1) / TOP).clamp(min=LEAST)
    return (x * (1.0 / scale)[:, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    T = case["T"]
    if case["op"] == "norm":
        H, D, dt = case["H"], case["D"], DT[case["dtype"]]
        # a few wide channels, rows of different size
        wide = 1.0 + 7.0 * (torch.rand(D, generator=g, device="cuda") < 0.01).float()
        size = torch.exp(0.5 * _normal(g, T, 1, 1))
        s["x"] = (_normal(g, T, H + case["gap"], D) * wide * size).to(dt)[:, :H]
        if case["add"]:
            s["add"] = _normal(g, T, H, D).to(dt)
            s["sum"] = torch.empty((T, H, D), dtype=dt, device="cuda")
        s["weight"] = ((1.0 - case["offset"] + 0.2 * _normal(g, D)).to(dt) if case["weight"]
                       else None)
        s["out"] = torch.empty((T, H, D), device="cuda",
                               dtype=torch.float8_e4m3fn if case["codes"] else dt)
        if case["codes"]:
            s["scales"] = torch.empty((T, H), device="cuda")
        return s
    if case["op"] == "route":
        E = case["E"]
        s["logits"] = 1.5 * _normal(g, T, E) + 0.5 * _normal(g, E)
        s["bias"] = 0.1 * _normal(g, E) if case["bias"] else None
        return s
    K, N, dt = case["K"], case["N"], DT[case["dtype"]]
    x = _normal(g, T, K + case["gap"])
    w = _normal(g, N, K) * K ** -0.5
    if case["dtype"] == "e4m3":
        s["x"], s["x_scale"] = _coded(x)
        s["w"], s["w_scale"] = _coded(w)
    else:
        s["x"], s["w"] = x.to(dt), w.to(dt)
    s["x"] = s["x"][:, :K]
    s["bias"] = 0.3 * _normal(g, N) if case["bias"] else None
    s["add"] = _normal(g, T, N).to(DT[case["out"]]) if case["add"] else None
    s["out"] = torch.empty((T, N), dtype=DT[case["out"]], device="cuda")
    return s


# ------------------------------------------------------------- plain form

def _normed(s):
    case = s["case"]
    x = s["x"].float()
    r = {}
    if case["add"]:
        x = x + s["add"].float()
        r["sum"] = x.to(s["x"].dtype)
    y = x * (1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + case["eps"]))
    if case["weight"]:
        y = y * (s["weight"].float() + case["offset"])
    elif case["offset"]:
        y = y * (1.0 + case["offset"])
    if not case["codes"]:
        r["out"] = y.to(s["x"].dtype)
        return r
    scale = (y.abs().amax(-1) / TOP).clamp(min=LEAST)
    r["out"] = (y * (1.0 / scale)[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    r["scales"] = scale
    return r


def _act(y, kind):
    if kind == "relu":
        return torch.where(y > 0, y, 0.0)
    if kind == "silu":
        return y / (1.0 + torch.exp(-y))
    if kind == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    return y


def _projected(s):
    case = s["case"]
    y = s["x"].float() @ s["w"].float().t()
    if case["dtype"] == "e4m3":
        y = y * (s["x_scale"][:, None] * s["w_scale"][None])
    if case["bias"]:
        y = y + s["bias"]
    y = _act(y, case["act"])
    if case["add"]:
        y = y + s["add"].float()
    return y.to(DT[case["out"]])


def _routed(s):
    case = s["case"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    dev = "cuda"
    # 64 bits: a choice between scores next to each other must not hang on rounding
    z = s["logits"].double()
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
    else:
        score = torch.exp(z - z.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    key = score + s["bias"].double() if case["bias"] else score
    if G > 1:
        per = key.view(T, G, E // G)
        rank = per.sort(dim=-1, descending=True).values[..., :case["best"]].sum(-1)
        order = rank.sort(dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        open_ = torch.zeros((T, G), dtype=torch.bool, device=dev).scatter_(1, order, True)
        key = torch.where(open_[..., None], per, -math.inf).view(T, E)
    ids = key.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    w = (w * case["factor"]).float()
    flat = ids.reshape(-1)
    perm = flat.sort(dim=0, stable=True).indices
    place = torch.arange(T * k, device=dev)
    inv = torch.empty_like(perm).scatter_(0, perm, place)
    counts = torch.zeros(E, dtype=torch.int64, device=dev).scatter_add_(
        0, flat, torch.ones_like(flat))
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device=dev), counts.cumsum(0)))
    blocks = (counts + BLOCK_M - 1) // BLOCK_M
    ends = blocks.cumsum(0)
    i = torch.arange(_most_tiles(case), device=dev)
    e = torch.searchsorted(ends, i, right=True).clamp(max=E - 1)
    within = (i - (ends - blocks)[e]) * BLOCK_M
    tiles = torch.stack((e, offsets[e] + within, (counts[e] - within).clamp(max=BLOCK_M)), -1)
    tiles = torch.where((i < ends[-1])[:, None], tiles, 0)
    r = dict(ids=ids, counts=counts, offsets=offsets, perm=perm, inv=inv, tiles=tiles,
             n_tiles=ends[-1:])
    return {**{n: v.int() for n, v in r.items()}, "w": w}


# -------------------------------------------------------- framework's calls

def _handles(s):
    """The structures a program keeps beside its tensors."""
    from routing_q4_grouped_gb300 import moeq4
    case, h = s["case"], {"moeq4": moeq4}
    if case["op"] == "linear":
        h["linear"] = moeq4.Linear(s["w"], bias=s["bias"], scale=s.get("w_scale"))
        h["act"] = {"none": moeq4.MOE_ACT_NONE, "relu": moeq4.MOE_ACT_RELU,
                    "silu": moeq4.MOE_ACT_SILU, "gelu": moeq4.MOE_ACT_GELU,
                    "gelu_tanh": moeq4.MOE_ACT_GELU_TANH}[case["act"]]
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        kind = {"softmax": moeq4.MOE_SCORE_SOFTMAX, "sigmoid": moeq4.MOE_SCORE_SIGMOID}
        h["spec"] = moeq4.RouteScore(kind[case["score"]], bias=s["bias"], groups=case["groups"],
                                     top_groups=case["top_groups"], group_best=case["best"],
                                     renorm=case["renorm"], factor=case["factor"])
        r = h["out"] = moeq4.RouteBuffers.alloc(T, E, k, BLOCK_M)
        r.tiles.zero_()                 # entries behind the map's end are left as they were
        h["ws"] = moeq4.alloc_workspace(moeq4.moe_route_workspace_size(T, E, k))
    return h


def _calls(s):
    case = s["case"]
    h = s.get("handles") or s.setdefault("handles", _handles(s))
    moeq4 = h["moeq4"]
    if case["op"] == "norm":
        r = {"out": s["out"]}
        kw = {}
        if case["add"]:
            kw.update(add=s["add"], sum=s["sum"])
            r["sum"] = s["sum"]
        if case["codes"]:
            kw.update(codes=s["out"], scales=s["scales"])
            r["scales"] = s["scales"]
        else:
            kw.update(out=s["out"])
        moeq4.moe_rms_norm(s["x"], s["weight"], eps=case["eps"], offset=case["offset"], **kw)
        return r
    if case["op"] == "linear":
        moeq4.moe_linear(s["x"], h["linear"], s["out"], act=h["act"], add=s["add"],
                         x_scale=s.get("x_scale"))
        return s["out"]
    r = h["out"]
    moeq4.moe_route_scored(s["logits"], h["spec"], r, h["ws"])
    return dict(ids=r.ids, w=r.w, counts=r.counts, offsets=r.offsets, perm=r.perm, inv=r.inv,
                tiles=r.tiles[:_most_tiles(case)], n_tiles=r.n_tiles[:1])


def run(state):
    if own:
        return _calls(state)
    return {"norm": _normed, "linear": _projected, "route": _routed}[state["case"]["op"]](state)


# ------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        r = {}
        if case["add"]:
            h = torch.add(h, s["add"].double())
            r["sum"] = h
        gain = 1.0 if s["weight"] is None else s["weight"].double()
        y = torch.rsqrt(torch.linalg.vector_norm(h, dim=-1, keepdim=True) ** 2 / case["D"]
                        + case["eps"]) * h * (gain + case["offset"])
        if not case["codes"]:
            return {**r, "out": y}
        top = torch.linalg.vector_norm(y, ord=math.inf, dim=-1)
        unit = torch.clamp(top / TOP, min=LEAST)
        return {**r, "out": y / unit[..., None], "scales": unit}
    if case["op"] == "linear":
        x, w = s["x"].double(), s["w"].double()
        if case["dtype"] == "e4m3":
            x = x * s["x_scale"].double()[:, None]
            w = w * s["w_scale"].double()[:, None]
        y = torch.einsum("tk,nk->tn", x, w)
        if case["bias"]:
            y += s["bias"].double()
        if case["act"] == "relu":
            y = y.clamp(min=0)
        elif case["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif case["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif case["act"] == "gelu_tanh":
            u = y + 0.044715 * y ** 3
            y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * u)
        return y + s["add"].double() if case["add"] else y
    # routing: the weights of the chosen experts, from one token's definition at a time
    E, per = case["E"], case["E"] // case["groups"]
    z = s["logits"].double()
    p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, -1)
    rank = p.clone() if s["bias"] is None else p + s["bias"].double()[None]
    if case["groups"] > 1:
        blocks = rank.reshape(-1, case["groups"], per)
        worth = torch.topk(blocks, min(case["best"], per), dim=-1).values.sum(-1)
        least = torch.topk(worth, case["top_groups"], dim=-1).values[:, -1:]
        shut = (worth < least).repeat_interleave(per, dim=1)
        rank = rank.masked_fill(shut, -math.inf)
    chosen = torch.topk(rank, case["k"], dim=-1).indices
    w = torch.take_along_dim(p, chosen, 1)
    if case["renorm"]:
        w = w / torch.sum(w, 1, keepdim=True)
    return dict(ids=None, counts=None, offsets=None, perm=None, inv=None, tiles=None,
                n_tiles=None, w=w * case["factor"])
