"""4-bit caches at the ends of their range: V rows up to the largest that an append writes, in the tile kernel."""
import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged4_ref import Step4
from paged_ref import compare

pytestmark = pytest.mark.gpu


def check(s, floor):
    """O and lse of all rows against 64 bits: weights in bf16 (2^-8) or f16 above `floor` of the largest, which counts the
    keys that a row sees by their own size."""
    O, lse = s.run()
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(s.ws) == fl.OK
    wO, wl, tO, tl = s.reference(2.0 ** -8)
    row, G = 0, s.H // s.Hkv
    for r, n in enumerate(s.q_len):
        kv = s.kv_len[r]
        for h in range(s.Hkv):
            _, V = s.rows_of(r, h)
            sums = torch.cat([V.new_zeros(1, s.d), V.abs().cumsum(0)])  # of the first keys
            sees = [max(0, kv - n + i + 1) if s.causal else kv for i in range(n)]
            tO[row:row + n, h * G:(h + 1) * G] += floor * sums[sees][:, None]
        row += n
    compare(O, wO, tO, "O")
    compare(lse, wl, tl, "lse")


def put(s, r, j, byte):
    """The V byte of token j of request r, all heads, with the block scales halved (E4M3: eight codes down): at most 1344 times
    its power of two, so that byte 244 stays below bf16's largest value."""
    page, off = s.table_host[r][j // s.ps], j % s.ps
    s.vb[page, :, off] = (s.vb[page, :, off].int() - 8).clamp(min=0).to(torch.uint8)
    s.vs[page, :, off] = byte


# f16 weights below their normal range: half a step, 2^-25 of a reference that the row's largest weight is at least 1 of
FLOOR = 2.0 ** -25


@pytest.mark.parametrize("d,H,Hkv,ps", [(128, 4, 1, 16), (64, 2, 2, 128)])
@pytest.mark.parametrize("byte", [191, 192, 235, 238, 239, 240, 241, 242, 243, 244])
def test_the_largest_values_stay_with_the_rows_that_see_them(byte, d, H, Hkv, ps):
    """The last token of a chunk (0 x inf must not reach the rows before it), and one in its middle."""
    for at in ([-1], [-90], [-1, -2, -150]):
        s = Step4([200, 150], [200, 700], H=H, Hkv=Hkv, d=d, ps=ps, seed=byte)
        for r in range(2):
            for j in at:
                put(s, r, s.kv_len[r] + j, byte)
        check(s, FLOOR)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("byte", [192, 244])
@pytest.mark.parametrize("first", [0, 300, 1100])
def test_usual_blocks_behind_a_large_value(first, byte, causal):
    """The tile goes on in another unit, its other parts do not: a context split over many workers, one of them with the row."""
    s = Step4([257, 40], [2500, 60], H=4, Hkv=2, d=128, ps=32, seed=first, causal=causal)
    put(s, 0, first, byte)
    check(s, FLOOR)


def test_large_and_small_values_in_turn():
    """Rows of all kinds of tiles, block after block: f16, bf16 for small rows, wide; a key that is not finite among them."""
    s = Step4([300], [1700], H=2, Hkv=1, d=128, ps=128, seed=5)
    for j, byte in ((40, 90), (300, 150), (500, 200), (640, 100), (900, 244), (1100, 230), (1650, 255)):
        put(s, 0, j, byte)
    O, lse = s.run()
    torch.cuda.synchronize()
    assert torch.isnan(O[250:].float()).all()
    put(s, 0, 1650, 127)  # rows before it do not see it: any value does for the definition
    wO, wl, tO, tl = s.reference(2.0 ** -8)
    _, V = s.rows_of(0, 0)
    sums = V.abs().cumsum(0)
    tO[:250] += FLOOR * sums[1400:1650][:, None]
    compare(O[:250], wO[:250], tO[:250], "O")
    compare(lse, wl, tl, "lse")


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("every,kv,q,H,Hkv,ps", [(128, 2500, 200, 2, 1, 16), (640, 6000, 140, 8, 2, 64), (10 ** 6, 20000, 130, 8, 8, 128)])
def test_many_small_weights_beside_a_dominant_key(every, kv, q, H, Hkv, ps, odd):
    """Keys that take nearly all weight and hold nothing (attention sinks); the others lie 2^-25 to 2^-29 below them and make
    up the result.  f16 weights: half a step, 2^-25, of a reference that the largest weight is at least 2^7 of.  odd: a
    key whose exponent byte a tile of f16 does not hold, every other block."""
    s = Step4([q], [kv], H=H, Hkv=Hkv, d=64, ps=ps, scale=1.0, seed=every)
    g = torch.Generator().manual_seed(kv)
    at = lambda j: (torch.tensor(s.table_host[0])[j // ps].cuda(), (j % ps).cuda())  # noqa: E731
    s.k.zero_()
    s.kb.fill_(0x38)  # 1
    s.ks.fill_(127)
    page, off = at(torch.arange(0, kv, every))
    s.k[page, :, off, 0] = 7  # 6 in the first channel
    # 6 q log2(e) from 25.1 to 29.4
    s.q_rows.copy_((2.9 + 0.5 * torch.rand(s.q_rows.shape, generator=g)).bfloat16())
    s.v.copy_(torch.tensor([0x12, 0x24, 0x46, 0x33], dtype=torch.uint8)[torch.randint(0, 4, s.v.shape, generator=g)])  # 0.5 to 4
    s.vb.fill_(0x38)
    s.vs.fill_(127)
    s.v[page, :, off] = 0
    if odd:
        j = torch.arange(57, kv, 256)
        p2, o2 = at(j)
        s.ks[p2, :, o2] = 100  # rows of zeros: the scores stay
    O, lse = s.run()
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(s.ws) == fl.OK
    wO, wl, tO, tl = s.reference(2.0 ** -11)
    for h in range(H):
        K, V = s.rows_of(0, h * Hkv // H)
        see = torch.arange(kv, device="cuda")[None] <= torch.arange(kv - q, kv, device="cuda")[:, None]
        x = torch.where(see, s.q.view(q, H, 64)[:, h].double() @ K.T, -torch.inf)
        p = torch.exp(x - x.amax(1, keepdim=True))
        tO[:, h] += 2.0 ** -32 * (see.double() @ V.abs()) / p.sum(1, keepdim=True)
    compare(O, wO, tO, "O")
    compare(lse, wl, tl, "lse")
