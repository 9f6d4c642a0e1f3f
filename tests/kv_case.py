"""Attention cases built and checked on the GPU in float64, for sizes that the numpy oracle
would take too long over. Shares no code with the product path."""
import torch

from routing_q4_grouped_gb300 import moeq4

GROUP = 64


def quantise(x, bits):
    """bf16 values x [...][D] (float64) -> codes, scale, bias of each group of 64 (float64)."""
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    levels = 2 ** bits - 1
    scale = ((hi - lo) / levels).float().bfloat16().double()
    safe = torch.where(scale > 0, scale, 1.0)
    code = torch.round((g - lo[..., None]) / safe[..., None]).clamp(0, levels)
    return torch.where(scale[..., None] > 0, code, 0.0).flatten(-2), scale, lo


class Case:
    """Contexts in shuffled pages; bytes of slots that hold no token read as NaN.

    shape(x, what, b): changes the tokens' float64 keys and values x [n][2][Hkv][D] of the
    prefix ("prefix") or of request b ("own") before they are quantised.
    words(scale, bias, what, b): changes [n][2][Hkv][D/64] scales and biases after it."""

    def __init__(self, seed, lens, Hq, Hkv, D, bits, P, prefix=0, nq=1, shape=None, words=None,
                 spare=2):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lens_, self.B, self.nq, self.Hq, self.Hkv = list(lens), len(lens), nq, Hq, Hkv
        self.D, self.bits, self.P, self.prefix = D, bits, P, prefix
        self.max_len = max(lens, default=0)
        per, pre = [-(-n // P) for n in lens], -(-prefix // P)
        total = sum(per) + pre + spare
        order = torch.randperm(total, generator=self.gen, device="cuda")
        row, nb = D * bits // 8, D // GROUP
        data = torch.full((total, 2, Hkv, P * (row + 4 * nb)), 255, dtype=torch.uint8, device="cuda")
        codes = data[..., :P * row].unflatten(-1, (P, row))
        word = data[..., P * row:].unflatten(-1, (P, 4 * nb))
        self.table = torch.full((self.B, max(1, max(per, default=0)) + 1), 0x7FFFFFFF,
                                dtype=torch.int32, device="cuda")
        self.kv, at = [], 0

        def fill(n, pages, what, b):
            x = torch.randn((n, 2, Hkv, D), generator=self.gen, device="cuda", dtype=torch.float64)
            if shape:
                shape(x, what, b)
            c, s, z = quantise(x.bfloat16().double(), bits)
            if words:
                words(s, z, what, b)
            t = torch.arange(n, device="cuda")
            q = c.to(torch.uint8)
            pg = pages[t // P]
            codes[pg, :, :, t % P] = q if bits == 8 else q[..., 0::2] | (q[..., 1::2] << 4)
            w = torch.stack((s.float().bfloat16(), z.float().bfloat16()), -1)
            word[pg, :, :, t % P] = w.view(torch.uint8).flatten(-2)
            s, z = s.float().bfloat16().double(), z.float().bfloat16().double()
            return (c.unflatten(-1, (-1, GROUP)) * s[..., None] + z[..., None]).flatten(-2)

        for b, n in enumerate(lens):
            pages = order[at:at + per[b]]
            at += per[b]
            self.table[b, :per[b]] = pages.int()
            self.kv.append(fill(n, pages, "own", b))
        pages = order[at:at + pre]
        self.ptable = pages.int() if prefix else None
        self.shared = fill(prefix, pages, "prefix", -1)
        self.seen_own = [torch.ones(n, dtype=torch.bool, device="cuda") for n in lens]
        self.q = torch.randn((self.B * nq, Hq, D), generator=self.gen, device="cuda").bfloat16()
        self.cache = moeq4.KVCache(data, P, Hkv, D, bits)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def rows_kernel(self, max_len=None):
        """1: the prefix, 2: the own tokens go to the kernel for many query rows."""
        return moeq4.moe_debug_kv_attention_rows(self.B, self.nq, self.Hq, self.Hkv, self.D,
                                                 self.max_len if max_len is None else max_len,
                                                 self.prefix)

    def run(self, q=None, out=None, max_len=None, scale=None, stream=None, ws=None):
        q = self.q if q is None else q
        m = self.max_len if max_len is None else max_len
        if out is None:
            out = torch.full_like(self.q, 5.0)
        if ws is None:
            ws = moeq4.alloc_workspace(moeq4.moe_kv_attention_workspace_size(
                self.B, self.nq, self.Hq, self.Hkv, self.D, m, self.prefix))
            ws.fill_(255)                                       # its contents do not matter
        moeq4.moe_kv_attention(q, self.cache, self.table, self.lens, m, out, ws, nq=self.nq,
                               prefix_table=self.ptable, prefix_len=self.prefix, scale=scale,
                               stream=stream)
        return out

    def reference(self, scale=None):
        """(o, spread, reach) [B*nq][Hq][D], [..][D], [..] in float64: the output (NaN where a
        seen key, or a seen value of the element's group, is NaN), sum_t p_t |v_t| and the
        largest |scale| * sum_d |q_d| |k_td| of the seen tokens."""
        scale = self.D ** -0.5 if scale is None else scale
        G = self.Hq // self.Hkv
        q = self.q.double().view(self.B, self.nq, self.Hkv, G, self.D)
        o, spread = torch.zeros_like(q), torch.zeros_like(q)
        reach = torch.zeros(q.shape[:-1], dtype=torch.float64, device="cuda")
        for b, n in enumerate(self.lens_):
            kv = torch.cat((self.shared, self.kv[b]))
            limit = self.prefix + (n - self.nq + 1 + torch.arange(self.nq, device="cuda")).clamp(min=0)
            t = torch.arange(kv.shape[0], device="cuda")
            there = torch.cat((torch.ones(self.prefix, dtype=torch.bool, device="cuda"), self.seen_own[b]))
            ok = ((t[None] < limit[:, None]) & there)[:, None].expand(-1, G, -1).reshape(self.nq * G, -1)
            for h in range(self.Hkv):
                k, v = kv[:, 0, h], kv[:, 1, h]
                bad_k, bad_v = k.isnan().any(-1), v.isnan()
                k, v = k.nan_to_num(0.0), v.nan_to_num(0.0)
                rows = q[b, :, h].reshape(-1, self.D)
                z = (scale * (rows @ k.T)).masked_fill(~ok, -torch.inf)
                any_ = ok.any(-1, keepdim=True)
                p = torch.where(any_, torch.softmax(torch.where(any_, z, 0.0), -1), 0.0)
                y = p @ v
                y[(ok & bad_k).any(-1)] = torch.nan
                y[(ok.double() @ bad_v.double()) > 0] = torch.nan
                o[b, :, h] = y.view(self.nq, G, -1)
                spread[b, :, h] = (p @ v.abs()).view(self.nq, G, -1)
                if kv.shape[0]:
                    r = (abs(scale) * (rows.abs() @ k.abs().T)).masked_fill(~ok, 0.0)
                    reach[b, :, h] = r.amax(-1).view(self.nq, G)
        shape = (self.B * self.nq, self.Hq)
        return o.view(*shape, -1), spread.view(*shape, -1), reach.view(*shape)

    def check(self, out, scale=None, keys=2.0 ** -9, weights=2.0 ** -9, norm=2.2e-3, err=0):
        """`keys`: relative error of a key operand against its token's size (a logit moves by
        at most keys * reach, a weight by twice that); `weights`: of weights, values, sums and
        partial results together; then bf16's rounding of the output (2^-8). `norm` bounds
        the error of each value group's elements as a whole: bf16 rounds with 1.7e-3 in the
        mean square, fp16 operands add below 3e-4 each."""
        o, spread, reach = self.reference(scale)
        got = out.double()
        assert torch.equal(got.isnan(), o.isnan())
        loose = torch.expm1(2 * keys * reach)[..., None] + weights
        fine = ~o.isnan()
        gap = ((got - o).abs() - 2.0 ** -8 * o.abs() - spread * loose - 1e-30)[fine]
        assert gap.numel() == 0 or gap.max() <= 0
        g, ref = (torch.where(fine, x, 0.0).unflatten(-1, (-1, GROUP)) for x in (got, o))
        for j in range(self.D // GROUP):
            size = ref[..., j, :].norm()
            miss = (g - ref)[..., j, :].norm()
            assert miss <= norm * size, (j, float(miss / size))
        assert moeq4.moe_get_device_error(self.cache) == err
