"""A plain model of serving from a paged cache, for the tests: lists for the
pages, 64-bit torch for the rows and the attention.  It shares no code with
the library."""
from __future__ import annotations

import math
import random

import torch

import precision_causal_attention_token_gb300 as fl

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2


def pages_of(n, ps):
    return -(-n // ps)


def model_plan(table, free, old, new, q, ps, T):
    """(table, free stack, slots) after the step; table: list of lists, free: list (the stack, top last)."""
    table, free = [list(r) for r in table], list(free)
    for r in range(len(q)):
        free += table[r][pages_of(new[r], ps):pages_of(old[r], ps)]
    for r in range(len(q)):
        for i in range(pages_of(old[r], ps), pages_of(new[r], ps)):
            table[r][i] = free.pop()
    slots = []
    for r in range(len(q)):
        for i in range(q[r]):
            pos = new[r] - q[r] + i
            slots.append(table[r][pos // ps] * ps + pos % ps if pos >= 0 else -1)
    return table, free, slots + [-1] * (T - len(slots))


def quantize_rows(x):
    """E4M3 codes and UE8M0 bytes of rows [..., d], from the definition in 64 bits."""
    x = x.double()
    top = x.abs().amax(-1)
    e = torch.full(top.shape, -127, dtype=torch.int32)
    for k in range(-127, 122):  # the smallest e with top <= 448 2^e
        e = torch.where(top > 448.0 * 2.0 ** k, torch.full_like(e, k + 1), e)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    y = torch.ldexp(x, -e[..., None])
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    y = torch.round(y / step) * step  # ties to even
    return y.float().to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def row_values(codes, scales):
    return torch.ldexp(codes.view(torch.float8_e4m3fn).double(), (scales.int() - 127)[..., None])


class Step:
    """One serving step on the GPU: lengths, shuffled pages, a cache, queries."""

    def __init__(self, q, kv, *, H=4, Hkv=2, d=128, ps=16, cache="bf16", causal=True, pad=0, seed=0, scale=0.0,
                 max_q=0, spare=3, strided=False, q_extra=0, fill=None, dev="cuda"):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.q_len, self.kv_len, self.ps, self.H, self.Hkv, self.d, self.causal = q, kv, ps, H, Hkv, d, causal
        self.dev, self.cache, self.n_req, self.T = dev, cache, len(q), sum(q) + pad
        self.scale = scale or 1.0 / math.sqrt(d)
        need = [pages_of(n, ps) for n in kv]
        self.max_pages, self.n_pages = max(need + [1]) + 2, sum(need) + spare
        ids = list(range(self.n_pages))
        random.Random(seed).shuffle(ids)
        # entries past a request's pages are out of range on purpose: they must not be read
        table = [[-(7 + r)] * self.max_pages for r in range(self.n_req)]
        for r in range(self.n_req):
            for i in range(need[r]):
                table[r][i] = ids.pop()
        self.spare_pages = ids
        i32 = dict(dtype=torch.int32, device=dev)
        self.cu_q = torch.tensor([sum(q[:i]) for i in range(self.n_req + 1)], **i32)
        self.kv = torch.tensor(kv, **i32)
        self.table_host = table
        self.table = torch.tensor(table, **i32)
        randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        shape = (self.n_pages, Hkv, ps, d)
        kf, vf = (randn(*shape) * torch.exp(0.4 * randn(self.n_pages, Hkv, ps, 1)) for _ in range(2))
        if cache == "bf16":
            k, v, self.ks, self.vs = kf.bfloat16(), vf.bfloat16(), None, None
        else:
            (k, ks), (v, vs) = quantize_rows(kf), quantize_rows(vf)
            self.ks, self.vs = ks.to(dev), vs.to(dev)
        if fill is not None:  # what earlier owners left in slots that hold no token
            used = torch.zeros(self.n_pages, ps, dtype=torch.bool)
            for r in range(self.n_req):
                for j in range(kv[r]):
                    used[table[r][j // ps], j % ps] = True
            free = ~used[:, None, :, None].expand(shape)
            if cache == "bf16":
                k[free], v[free] = fill, fill
            else:
                k[free], v[free] = 0x7F, 0x7F
                self.ks[free[..., 0].to(dev)] = 255
                self.vs[free[..., 0].to(dev)] = 255
        if strided:  # K and V pages interleaved in one buffer
            both = torch.stack([k, v], 1).to(dev)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = k.to(dev), v.to(dev)
        self.q_rows = torch.zeros(self.T, H * d + q_extra, dtype=torch.bfloat16)
        self.q_rows[:, :H * d] = (1.5 * randn(self.T, H * d)).bfloat16()
        self.q_rows = self.q_rows.to(dev)
        self.q = self.q_rows[:, :H * d]
        self.prob = fl.make_paged(self.T, H, Hkv, d, self.cu_q, self.kv, self.table, page_size=ps,
                                  n_pages=self.n_pages, max_q=max_q, causal=causal, softmax_scale=scale,
                                  cache_dtype=fl.BF16 if cache == "bf16" else fl.E4M3,
                                  q_stride=H * d + q_extra if q_extra else 0)
        self.ws = torch.full((max(16, fl.flamia_paged_workspace_size(self.prob)),), 0xA5, dtype=torch.uint8, device=dev)
        self.pool = fl.paged_cache(self.k, self.v, self.ks, self.vs)

    def run(self, stream=None):
        self.O = torch.full((self.T, self.H, self.d), 77.0, dtype=torch.bfloat16, device=self.dev)
        self.lse = torch.full((self.H, self.T), 77.0, device=self.dev)
        fl.flamia_paged_plan(self.prob, self.ws, stream=stream)
        fl.flamia_paged_fwd(self.prob, self.q, self.pool, self.O, self.lse, self.ws, stream=stream)
        return self.O, self.lse

    def rows_of(self, r, h):
        """K, V [kv_len, d] of request r and key/value head h, in 64 bits."""
        n = self.kv_len[r]
        j = torch.arange(n)
        page = torch.tensor(self.table_host[r])[j // self.ps].to(self.dev)
        off = (j % self.ps).to(self.dev)
        k, v = self.k[page, h, off], self.v[page, h, off]
        if self.cache == "bf16":
            return k.double(), v.double()
        return row_values(k, self.ks[page, h, off]), row_values(v, self.vs[page, h, off])

    def reference(self, weight_rounding, weight_floor=0.0):
        """O, lse in 64 bits and how far a result may be from them.

        O: half a bf16 step of the value, plus what errs in the weights: their own rounding (`weight_rounding`
        relative, 0 where a second term holds what the first lost) and that of the scores in fp32.  A score is a sum
        of d products, each step of which rounds by at most 2^-23 of what is summed in magnitude (2^-23, not 2^-24:
        the matrix units may truncate); scaling, the subtraction of the reference and the exponential add 2^-22 of
        the score's size and of the result.

        weight_floor: E4M3 weights kept in f16 as p 2^(e - E + 7) (p: relative to a reference that the sum is at least
        1 of; e: the key's exponent, E: the largest) round by at most 2^-25 below f16's normal range, that is by 2^-32
        of 2^E times the code, at most 448: weight_floor = 2^-32 for each of the keys."""
        T, H, d, G = self.T, self.H, self.d, self.H // self.Hkv
        O = torch.full((T, H, d), 77.0, dtype=torch.float64, device=self.dev)
        lse = torch.full((H, T), 77.0, dtype=torch.float64, device=self.dev)
        tO, tl = torch.zeros_like(O), torch.zeros_like(lse)
        row = 0
        for r, n in enumerate(self.q_len):
            kv = self.kv_len[r]
            at = slice(row, row + n)
            row += n
            if not n:
                continue
            for h in range(self.Hkv):
                K, V = self.rows_of(r, h)
                for hq in range(h * G, (h + 1) * G):
                    Q = self.q[at].view(n, H, d)[:, hq].double()
                    last = torch.arange(n, device=self.dev) + (kv - n) if self.causal else torch.full((n,), kv - 1, device=self.dev)
                    see = torch.arange(kv, device=self.dev)[None, :] <= last[:, None]
                    x = torch.where(see, (Q @ K.T) * self.scale, -math.inf)
                    size = torch.where(see, (Q.abs() @ K.abs().T) * self.scale, 0.0)
                    m = x.amax(1, keepdim=True) if kv else torch.full((n, 1), -math.inf, device=self.dev, dtype=torch.float64)
                    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
                    s = p.sum(1, keepdim=True)
                    w = p / torch.where(s > 0, s, 1.0)
                    O[at, hq] = w @ V
                    lse[hq, at] = (m + s.log())[:, 0]
                    err = size * (d + 4) * 2.0 ** -23 + 2.0 ** -21  # of a score, and so relative of a weight
                    rel = (w * err).sum(1, keepdim=True)  # of the sum
                    A = (w * (err + weight_rounding)) @ V.abs() + rel * (w @ V.abs())
                    low = weight_floor * kv * 448.0 * float(self.largest_scale(r, h)) if weight_floor and kv else 0.0
                    tO[at, hq] = HALF_BF16 * O[at, hq].abs() + 1.02 * A + low + 2.0 ** -126
                    tl[hq, at] = rel[:, 0] * 1.02 + 2.0 ** -22 * lse[hq, at].abs().nan_to_num(0, 0, 0) + 2.0 ** -20
        return O, lse, tO, tl

    def largest_scale(self, r, h):
        j = torch.arange(self.kv_len[r])
        page = torch.tensor(self.table_host[r])[j // self.ps].to(self.dev)
        b = self.vs[page, h, (j % self.ps).to(self.dev)].int()
        return 2.0 ** (int(b[b != 255].max()) - 127)

    def rounding(self):
        """(weight_rounding, weight_floor): the tile kernel rounds the weights to bf16, the decode kernel to two bf16
        terms over a bf16 cache and to f16 over an E4M3 one."""
        if self.chunk_path():
            return HALF_BF16, 0.0
        return (HALF_BF16 ** 2, 0.0) if self.cache == "bf16" else (torch.finfo(torch.float16).eps / 2, 2.0 ** -32)

    def chunk_path(self):
        return (max(1, self.prob.max_q or self.T)) * (self.H // self.Hkv) > 32

    def check(self):
        O, lse = self.run()
        torch.cuda.synchronize()
        st = fl.flamia_get_device_status(self.ws)
        assert st == fl.OK, fl.status_string(st)
        wO, wl, tO, tl = self.reference(*self.rounding())
        compare(O, wO, tO, "O")
        compare(lse, wl, tl, "lse")


def compare(got, want, tol, what):
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), f"{what}: other values are infinite or NaN"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    err = (got - want).abs()[fine]
    over = err - tol[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, (
        f"{what}: off by {float(err[over.argmax()]):.3e} where {float(tol[fine][over.argmax()]):.3e} is allowed "
        f"({int((over > 0).sum())} of {over.numel()})")
