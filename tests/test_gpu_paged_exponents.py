"""E4M3 caches whose rows have scales of very different size: what lies behind
the last token, tokens that a row may not see, rows of zeros and keys of no
weight must not cost the others their bits."""
import math

import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged_ref import Step, compare

pytestmark = pytest.mark.gpu

# The decode kernel's weight p of a key (p: relative to a reference that the row's sum is at least 1 of) is kept in f16
# as p 2^(e - E + 7), E the largest of the key exponents that a warp has met and at most 12 above e: half a step of
# f16's smallest numbers, 2^-25, is 2^(-25 - 7 + 12) of p.  Warps whose exponents lie farther apart hold two bf16 terms.
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
            sums = torch.cat([V.new_zeros(1, s.d), V.abs().cumsum(0)])  # of the first keys
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


def put(s, r, j, byte, codes=None):
    """The V byte (and codes) of token j of request r, all heads."""
    page, off = s.table_host[r][j // s.ps], j % s.ps
    s.vs[page, :, off] = byte
    if codes is not None:
        s.v[page, :, off] = codes


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


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("above", [12, 13, 24, 40, 90])
def test_a_later_tokens_size(kind, d, above):
    """A large V row of a later new token leaves the rows before it as they are."""
    s = step(kind, d=d, ps=32, seed=3)
    s.vs.fill_(120)
    for r in (0, 2, 3):
        put(s, r, KV[r] - 1, 120 + above)
    check(s)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("small", [10, 33, 80])
def test_rows_of_zeros_beside_small_ones(kind, d, small):
    """A row of zeros is stored under byte 127, however small the others are."""
    s = step(kind, d=d, ps=16, seed=5)
    s.vs -= small
    for r, j in ((0, 0), (0, 20), (2, 64), (3, 200), (4, 1)):
        put(s, r, j, 127, 0)
    check(s)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spread", [13, 40, 180])
def test_sizes_far_apart_and_peaked_rows(kind, d, spread):
    """V rows over many binades, and softmax rows that give most of them no weight to speak of."""
    s = step(kind, d=d, ps=16, seed=9, scale=1.5)
    g = torch.Generator().manual_seed(11)
    b = torch.randint(128 - spread // 2, 129 + spread // 2, s.vs.shape, generator=g)
    s.vs.copy_(b.to(torch.uint8))
    check(s)


@pytest.mark.parametrize("H", [8, 16, 32])
def test_sizes_far_apart_over_a_split_context(H):
    """Small rows first, large ones late, over many workers and warps; a NaN row in the other head only."""
    s = Step([1], [9001], H=H, Hkv=1, ps=64, cache="e4m3", seed=H, max_q=1)
    for at, byte in ((0, 60), (5, 60), (3000, 150), (8999, 190)):
        put(s, 0, at, byte)
    check(s)


@pytest.mark.parametrize("q", [2, 4, 8])
def test_a_nan_row_beside_sizes_far_apart(q):
    """Byte 255 in a warp that takes its keys carefully: NaN for the rows that see it, the others keep their values."""
    s = Step([q], [100], H=4, Hkv=1, ps=32, cache="e4m3", seed=q, max_q=q)
    put(s, 0, 3, 180)
    put(s, 0, 99 - (q - 1) // 2, 125)
    wO, wl, tO, tl = s.reference(2.0 ** -11)
    _, V = s.rows_of(0, 0)
    tO += FLOOR * V.abs().sum(0)
    put(s, 0, 99 - (q - 1) // 2, 255, 0x7F)
    O, lse = s.run()
    first = q - 1 - (q - 1) // 2  # the first row that sees it
    assert torch.isnan(O[first:]).all()
    compare(O[:first], wO[:first], tO[:first], "O")
    compare(lse, wl, tl, "lse")
    assert math.isfinite(float(lse.abs().max()))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("up", [115, 60, -60, -115])
def test_large_keys_and_small_queries(kind, d, up):
    """Keys of 2^115 against queries of 2^-115, and the other way: the scores are ordinary numbers."""
    s = step(kind, d=d, ps=16, seed=13)
    s.ks += up
    s.q_rows.copy_((s.q_rows.float() * 2.0 ** -up).bfloat16())
    check(s)
