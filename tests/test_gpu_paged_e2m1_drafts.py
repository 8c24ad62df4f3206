"""4-bit caches, V rows up to the largest that an append writes beside usual ones: few query rows (the pass that takes a
warp's keys once more, with bf16 values) and a chunk."""
import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged4_ref import Step4, packed, quantize4
from paged_ref import compare
from test_gpu_paged_e2m1_sizes import check, put

pytestmark = pytest.mark.gpu

# f16 weights: p 2^(e - E + 7), E at most 12 above e (farther: two bf16 terms); half a step, 2^-25, is 2^-20 of p
FLOOR = 2.0 ** -20
KINDS = {"8 rows": dict(q=[4, 2], H=2), "16 rows": dict(q=[4, 3], H=4), "32 rows": dict(q=[8, 5], H=4), "one": dict(q=[1, 1], H=8), "chunk": dict(q=[150, 60], H=2)}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("byte", [150, 192, 235, 240, 242, 243, 244])
def test_the_largest_values_stay_with_the_rows_that_see_them(byte, d, kind):
    k = KINDS[kind]
    for at in ([-1], [-40], [-1, -2, -190]):
        s = Step4(k["q"], [200, 900], H=k["H"], Hkv=1, d=d, ps=16, max_q=max(k["q"]), seed=byte)
        for r in range(2):
            for j in at:
                put(s, r, s.kv_len[r] + j, byte)
        check(s, FLOOR)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_the_largest_finite_numbers(kind, d):
    """A row of bf16's largest value is stored as 2^128 and a little: infinite in 16 and 32 bits.  It is the result of rows
    that give it all their weight, and nothing of those that do not see it."""
    k = KINDS[kind]
    n = max(k["q"])
    s = Step4([n], [300], H=k["H"], Hkv=1, d=d, ps=16, max_q=n)
    page, off = s.table_host[0][299 // 16], 299 % 16
    c, b, e = quantize4(torch.full((d,), torch.finfo(torch.bfloat16).max, dtype=torch.float64))
    s.v[page, 0, off], s.vb[page, 0, off], s.vs[page, 0, off] = packed(c).cuda(), b.cuda(), int(e)
    wO, wl, tO, tl = s.reference(2.0 ** -8)
    V = s.rows_of(0, 0)[1]
    assert float(V[-1].min()) > 2.0 ** 128
    sums = V.abs().cumsum(0)
    for i in range(n):
        tO[i] += FLOOR * sums[300 - n + i]
    O, lse = s.run()
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(s.ws) == fl.OK
    sure = wO.abs() + tO < float(torch.finfo(torch.bfloat16).max)  # else the infinity of its sign does as well
    compare(torch.where(sure, O.double(), 0.0), torch.where(sure, wO, 0.0), tO, "O")
    assert sure[:-1].all() and (O[~sure].double() > 2.0 ** 127).all()
    compare(lse, wl, tl, "lse")


@pytest.mark.parametrize("q,max_q,H", [([4, 2], 4, 2), ([4, 3], 4, 4), ([8, 5], 8, 4), ([1, 1], 1, 8), ([150, 90], 0, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_every_row_large(q, max_q, H, d):
    """Means that fit where the sums of their terms would not: rows of 2^122 and more, weights nearly equal."""
    Step = lambda **kw: Step4(q, [200, 900], H=H, Hkv=1, d=d, ps=32, max_q=max_q, scale=0.02,  # noqa: E731
                              shift=lambda *s: torch.full(s, 122), **kw)
    s = Step()
    assert int(s.vs.max()) < 244 and float(s.rows_of(1, 0)[1].abs().max()) < 2.0 ** 128
    check(s, FLOOR)
    s = Step(seed=3)
    s.vs[s.table_host[1][0], :, 0] = 127  # and one of the usual size: the careful pass
    check(s, FLOOR)
