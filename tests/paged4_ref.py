"""The 4-bit cache (E2M1 codes, E4M3 block scales, a power-of-two row exponent) from its definition, for the tests."""
from __future__ import annotations

import torch

import precision_causal_attention_token_gb300 as fl
from paged_ref import Step, HALF_BF16

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # its values from 0 up to 448


def quantize4(x):
    """codes [..., d] (0..15), block scale bytes [..., d / 16], exponent bytes [...] of rows, by searching the values in
    64 bits; rows that are not finite are zeros under byte 255."""
    x = x.double()
    finite = torch.isfinite(x).all(-1)
    x = torch.where(finite[..., None], x, 0.0)
    top = x.abs().amax(-1)
    e = torch.full(top.shape, -127, dtype=torch.int32)
    for k in range(-127, 120):  # the smallest e with top <= 2688 2^e
        e = torch.where(top > 2688.0 * 2.0 ** k, torch.full_like(e, k + 1), e)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    y = torch.ldexp(x, -e[..., None]).unflatten(-1, (-1, 16))
    block = torch.searchsorted(6.0 * E4M3, y.abs().amax(-1))  # the first with 6 s >= the maximum
    s = E4M3[block]
    z = torch.where(s[..., None] > 0, y / torch.where(s > 0, s, 1.0)[..., None], 0.0)
    d = (z.abs()[..., None] - LEVELS).abs()
    near = d.amin(-1, keepdim=True)
    even = torch.arange(8) % 2 == 0
    code = torch.where(d == near, torch.where(even, 0, 1), 2).argmin(-1)  # of two nearest the even one
    code = torch.where(z < 0, code + 8, code)
    return code.flatten(-2).to(torch.uint8), block.to(torch.uint8), torch.where(finite, e + 127, 255).to(torch.uint8)


def packed(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def unpacked(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def values4(codes, blocks, scales):
    """Packed rows -> 64 bits; byte 255 is NaN."""
    level = torch.cat([LEVELS, -LEVELS]).to(codes.device)
    v = level[unpacked(codes).long()].unflatten(-1, (-1, 16)) * blocks.view(torch.float8_e4m3fn).double()[..., None]
    v = torch.ldexp(v.flatten(-2), (scales.int() - 127)[..., None])
    return torch.where((scales == 255)[..., None], torch.nan, v)


class Step4(Step):
    """A serving step over a 4-bit cache.  shift(n_pages, Hkv, ps) -> exponents added to the rows of V; k_shift: to the
    rows of K, and taken from the queries."""

    def __init__(self, q, kv, *, strided=False, poison=False, shift=None, k_shift=0, **kw):
        super().__init__(q, kv, cache="bf16", **kw)
        dev = self.dev
        kf, vf = self.k.cpu(), self.v.cpu()
        parts = [quantize4(kf), quantize4(vf)]
        codes, blocks, scales = ([p[i] for p in parts] for i in range(3))
        codes = [packed(c) for c in codes]
        if shift is not None:
            scales[1] = (scales[1].int() + shift(*scales[1].shape)).clamp(0, 254).to(torch.uint8)
        if k_shift:
            scales[0] = (scales[0].int() + k_shift).clamp(0, 254).to(torch.uint8)
            self.q_rows.copy_((self.q_rows.double() * 2.0 ** -k_shift).bfloat16())
        if poison:  # what earlier owners left in slots that hold no token
            free = torch.ones(self.n_pages, self.ps, dtype=torch.bool)
            for r in range(self.n_req):
                for j in range(kv[r]):
                    free[self.table_host[r][j // self.ps], j % self.ps] = False
            free = free[:, None].expand(scales[0].shape)
            for i in range(2):
                codes[i][free], blocks[i][free], scales[i][free] = 0xF7, 0x7F, 255
        if strided:
            both = torch.stack(codes, 1).to(dev)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = (c.to(dev) for c in codes)
        self.kb, self.vb = (b.to(dev) for b in blocks)
        self.ks, self.vs = (s.to(dev) for s in scales)
        self.cache = "e2m1"
        self.prob.cache_dtype = fl.E2M1
        self.pool = fl.paged_cache(self.k, self.v, self.ks, self.vs, self.kb, self.vb)

    def rows_of(self, r, h):
        j = torch.arange(self.kv_len[r])
        page = torch.tensor(self.table_host[r])[j // self.ps].to(self.dev)
        off = (j % self.ps).to(self.dev)
        return tuple(values4(c[page, h, off], b[page, h, off], s[page, h, off])
                     for c, b, s in ((self.k, self.kb, self.ks), (self.v, self.vb, self.vs)))

    def rounding(self):
        """As over an E4M3 cache, but that a value is up to 6 * 448 of its row's power of two, in place of 448, and that the
        tile kernel's weights are f16 where all of V's exponent bytes are 112 to 127: off by 2^-25 of a reference that the
        sum is at least 1 of below f16's normal range."""
        half = torch.finfo(torch.float16).eps / 2
        if not self.chunk_path():
            return half, 6.0 * 2.0 ** -32
        used = [self.vs[self.table_host[r][j // self.ps], :, j % self.ps] for r in range(self.n_req) for j in range(self.kv_len[r])]
        used = torch.stack(used) if used else torch.full((1,), 127)
        return (half, 6.0 * 2.0 ** -25) if int(used.min()) >= 112 and int(used.max()) <= 127 else (HALF_BF16, 6.0 * 2.0 ** -25)
