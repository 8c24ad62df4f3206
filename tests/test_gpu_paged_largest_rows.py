"""An E4M3 cache with a row of bf16's largest number, which is stored as 256 * 2^120: infinite in 16 and in 32 bits."""
import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged_ref import Step, compare, quantize_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q,H", [([4], 2), ([4], 4), ([8], 4), ([150], 2)])
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 128)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_row_of_the_largest_number_stays_with_those_that_see_it(q, H, d, ps, sign):
    n = q[0]
    s = Step(q, [300], H=H, Hkv=1, d=d, ps=ps, cache="e4m3", max_q=n, seed=d)
    page, off = s.table_host[0][299 // ps], 299 % ps
    code, byte = quantize_rows(torch.full((d,), sign * torch.finfo(torch.bfloat16).max, dtype=torch.float64))
    s.v[page, 0, off], s.vs[page, 0, off] = code.cuda(), int(byte)
    V = s.rows_of(0, 0)[1]
    assert float(V[-1].abs().min()) == 2.0 ** 128
    O, lse = s.run()
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(s.ws) == fl.OK
    wO, wl, tO, tl = s.reference(2.0 ** -8)
    sums = V.abs().cumsum(0)
    for i in range(n):
        tO[i] += 2.0 ** -20 * sums[300 - n + i]  # f16 weights: 2^-20 of the largest
    compare(O[:-1], wO[:-1], tO[:-1], "O")  # the last row's sum passes fp32
    compare(lse, wl, tl, "lse")
