"""Shared pages: a free stack with an entry outside the pool."""
import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged_pages_ref import Pool
from test_gpu_paged_pages import Gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("entry", [12, -1, 1 << 30, -(1 << 31)])
@pytest.mark.parametrize("at", [-1, -2])
def test_a_step_refuses_to_take_a_page_outside_the_pool(at, entry):
    """Of the two pages that the step takes (a copy on write, a longer row): nothing moves, and with the entry put right the
    same step goes through."""
    m = Pool(3, 12, 4, 16)
    gpu = Gpu(m, 3, 64, 40)
    m.step([20, 40, 0], [20, 40, 0], [0, 1, 2])
    gpu.inputs([20, 40, 0], [20, 40, 0], [0, 1, 2], [0, 0, 0])
    assert gpu.step() == fl.OK
    q, kv, src = [1, 1, 9], [21, 21, 49], [0, 0, 1]
    gpu.inputs(q, kv, src, m.held)
    at = at % len(m.free)
    gpu.free[at] = entry
    state = (gpu.table, gpu.refs, gpu.free, gpu.n_free)
    before = [x.clone() for x in state]
    gpu.n_copies.fill_(5)
    assert gpu.step() == fl.ERR_BAD_PAGE == fl.flamia_get_device_status(gpu.pages_ws)
    assert all(torch.equal(a, b) for a, b in zip(state, before))
    assert (gpu.slots == -1).all() and int(gpu.n_copies) == 0
    gpu.free[at] = m.free[at]
    copies = m.step(q, kv, src)
    assert len(copies) == 1 and gpu.step() == fl.OK
    gpu.same(copies)
    assert gpu.slots.tolist() == m.slots(q, kv, 64)


def test_a_long_row_takes_no_page_outside_the_pool():
    """Thousands of pages for one row, a bad one anywhere among them."""
    m = Pool(2, 5000, 4000, 16)
    gpu = Gpu(m, 2, 64000, 64000)
    for at in (4999, 4998, 3000, 1500, 1002):  # the row takes 3,999 pages
        gpu.inputs([63970, 0], [63970, 0], [0, 1], [0, 0])
        gpu.free[at] = 5000
        assert gpu.step() == fl.ERR_BAD_PAGE and int(gpu.refs.sum()) == 0 and int(gpu.table.abs().sum()) == 0
        gpu.free[at] = at
    gpu.free[1000] = -3  # left on the stack
    copies = m.step([63970, 0], [63970, 0], [0, 1])
    m.free[1000] = -3
    assert gpu.step() == fl.OK
    gpu.same(copies)


def test_entries_behind_the_count_are_not_read():
    m = Pool(200, 900, 4, 16)
    gpu = Gpu(m, 200, 400, 2)
    for it in range(3):
        q, kv = [2] * 200, [2 + 2 * it] * 200
        gpu.inputs(q, kv, list(range(200)), m.held)
        copies = m.step(q, kv, list(range(200)))
        gpu.free[int(gpu.n_free):] = -7
        assert gpu.step() == fl.OK
        gpu.same(copies)
