"""Rows appended to a 4-bit cache, K and V, whose blocks differ by more than fp32's range of exponents."""
import pytest
import torch

from paged4_ref import packed, quantize4
from test_gpu_paged_e2m1 import _append, _same_rows

pytestmark = pytest.mark.gpu


def _compare(got, rows):
    for (c, b, s), r in zip(got, rows):
        wc, wb, ws = quantize4(r)
        assert torch.equal(s.cpu(), ws) and torch.equal(b.cpu(), wb)
        _same_rows(c, packed(wc), "codes")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_blocks_far_below_their_rows(dtype, d):
    """A block that is not zero has a scale that is not zero, however far it lies below the row's largest element."""
    tiny = [2.0 ** -133, 2.0 ** -126, 1e-38, 1e-30, 1e-20, 2.0 ** -30, 2.0 ** -21, 2.0 ** -20]
    if dtype == torch.float32:
        tiny += [2.0 ** -149, 2.0 ** -148, 2.0 ** -140]
    rows = []
    for top in (3e38, 1.5e38, 1e30, 2.0 ** 40, 2688.0, 1.0, 2.0 ** -60, 2.0 ** -115, 2.0 ** -120):
        for x in tiny:
            for sign in (1.0, -1.0):
                row = torch.zeros(d, dtype=torch.float64)
                row[0], row[16 + 5], row[32] = top / 2, sign * x, -x
                rows.append(row)
    x = torch.stack(rows).to(dtype)[:, None]
    got, rows = _append(torch.cat([x, x.flip(0)], 1), d, dtype, 64)
    assert (got[0][1] == 1).any()  # the smallest block scale
    _compare(got, rows)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_borders_between_codes_in_v(dtype):
    """Every border between two codes and its neighbours under every block scale, as K and, doubled, as V."""
    tie = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
    rows = []
    for code in range(1, 127):
        s = torch.tensor([code], dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        row = torch.zeros(8, 16, dtype=torch.float64)
        row[0, 0] = 2688.0  # exponent 0
        for i, f in enumerate((1.0, 1 + step, 1 - step, 1 + 2 * step, -1.0, -1 - step)):
            row[1 + i, :7] = tie * s * f
            row[1 + i, 15] = 6 * s
        rows.append(row.flatten())
    x = torch.stack(rows).to(dtype)
    x = torch.cat([x, (x.double() * 2.0 ** -100).to(dtype), (x.double() * 2.0 ** 90).to(dtype)])[:, None]
    _compare(*_append(torch.cat([x, x.flip(0)], 1), 128, dtype, 64))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_that_are_not_finite_in_v(dtype):
    """2 x is infinite where x is finite: V's row is marked, K's is not."""
    x = torch.zeros(4, 1, 64)
    x[0, 0, 3], x[1, 0, 3], x[1, 0, 40], x[2, 0, 9], x[3, 0, 63] = 3e38, -3e38, 1e-30, 1.6e38, float("nan")
    got, rows = _append(x, 64, dtype, 16)
    assert got[0][2].flatten().tolist()[3] == 255 and got[1][2].flatten().tolist()[:2] == [255, 255]
    for (c, b, s), r in zip(got, rows):
        wc, wb, ws = quantize4(r)
        fine = (ws != 255)
        assert torch.equal(s.cpu(), ws) and torch.equal(b.cpu()[fine], wb[fine])
        _same_rows(c[fine.cuda()], packed(wc)[fine], "codes")
