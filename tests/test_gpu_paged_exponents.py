"""E4M3 caches whose rows have scales of very different size: what lies behind
the last token must not cost the others their bits."""
import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged_ref import Step, compare

pytestmark = pytest.mark.gpu

# The decode kernel's weight p of a key (p: relative to a reference that the row's sum is at least 1 of) is kept in f16
# as p 2^(e - E + 7), E the largest of the key exponents that a warp has met, here at most 12 above e: half a step of
# f16's smallest numbers, 2^-25, is 2^(-25 - 7 + 12) of p.
FLOOR = 2.0 ** -20


def check(s):
    """O and lse of all rows against 64 bits; the weights' floor counts the keys that a row sees, by their own size."""
    O, lse = s.run()
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(s.ws) == fl.OK
    wO, wl, tO, tl = s.reference(2.0 ** -8 if s.chunk_path() else 2.0 ** -11)
    row, G = 0, s.H // s.Hkv
    for r, n in enumerate(s.q_len):
        kv = s.kv_len[r]
        for h in range(s.Hkv):
            _, V = s.rows_of(r, h)
            sums = torch.cat([torch.zeros_like(V[:1]), V.abs().cumsum(0)])  # of the first keys
            sees = [max(0, kv - n + i + 1) if s.causal else kv for i in range(n)]
            tO[row:row + n, h * G:(h + 1) * G] += FLOOR * sums[sees][:, None]  # few rows: also in a call with chunks
        row += n
    compare(O, wO, tO, "O")
    compare(lse, wl, tl, "lse")


def free_slots(s):
    used = torch.zeros(s.n_pages, s.ps, dtype=torch.bool)
    for r in range(s.n_req):
        for j in range(s.kv_len[r]):
            used[s.table_host[r][j // s.ps], j % s.ps] = True
    return ~used[:, None, :].expand(-1, s.Hkv, -1)


# rows of a key/value head: 8, 16 and 32 in the decode kernel, then a chunk with decoding requests
KINDS = {"8 rows": dict(q=[2, 1, 2, 2, 1], H=8), "16 rows": dict(q=[4, 1, 3, 4, 2], H=8),
         "32 rows": dict(q=[8, 1, 5, 7, 3], H=8), "chunk": dict(q=[40, 1, 30, 140, 5], H=8)}
KV = [45, 1, 131, 333, 5]


def step(kind, **kw):
    k = KINDS[kind]
    return Step(k["q"], kw.pop("kv", KV), H=k["H"], Hkv=2, cache="e4m3", max_q=max(k["q"]), **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("byte", [147, 200, 254, -1])
def test_bytes_behind_the_last_token(kind, d, byte):
    """Large finite scale bytes (or any, -1) and any codes in slots that hold no token: earlier owners' or fresh memory."""
    for ps in (16, 128):
        s = step(kind, d=d, ps=ps, seed=d + ps)
        g = torch.Generator().manual_seed(7)
        free = free_slots(s)
        for codes, scales in ((s.k, s.ks), (s.v, s.vs)):
            b = torch.randint(0, 256, scales.shape, generator=g) if byte < 0 else torch.full(scales.shape, byte)
            c = torch.randint(0, 256, codes.shape, generator=g)
            scales[free] = b[free].to(torch.uint8).cuda()
            codes[free] = c[free].to(torch.uint8).cuda()
        check(s)
