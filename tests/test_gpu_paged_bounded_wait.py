"""The page calls' barriers over their CTAs are bounded waits.  A test hook keeps one CTA away from a launch's last one: the
wait runs out, every CTA leaves, no page moves, the status says so, and the same buffers serve the next call."""
import contextlib

import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged_pages_ref import Pool
from test_gpu_paged_pages import Gpu

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def withheld():
    fl.flamia_debug_withhold_first_item(True)
    try:
        yield
    finally:
        fl.flamia_debug_withhold_first_item(False)


def _held(n):
    """n requests of different lengths whose pages lie anywhere in the pool; every third has ended."""
    m = Pool(n, 8 * n + 20, 6, 16)
    gpu = Gpu(m, n, 64 * n, 64)
    for kv in ([20 + 7 * i % 40 for i in range(n)], [0 if i % 3 == 0 else 20 + 7 * i % 40 for i in range(n)]):
        q = kv if not any(m.held) else [0] * n
        gpu.inputs(q, kv, list(range(n)), m.held)
        m.step(q, kv, list(range(n)))
        assert gpu.step() == fl.OK
    gpu.old.copy_(torch.tensor(m.held, dtype=torch.int32))
    return m, gpu


def _state(gpu):
    return [x.clone() for x in (gpu.table, gpu.refs, gpu.free, gpu.n_free)]


@pytest.mark.parametrize("n", [1, 7, 400])
def test_a_compaction_whose_wait_runs_out_moves_nothing(n):
    m, gpu = _held(n)
    before = _state(gpu)
    gpu.n_copies.fill_(9)
    with withheld():
        assert gpu.compact() == fl.ERR_TIMEOUT
    assert all(torch.equal(a, b) for a, b in zip(_state(gpu), before)) and int(gpu.n_copies) == 0
    moves = m.compact()
    assert gpu.compact() == fl.OK
    gpu.same(moves)


@pytest.mark.parametrize("n", [1, 7, 400])
def test_a_step_whose_wait_runs_out_moves_nothing(n):
    m, gpu = _held(n)
    src = [(i + 1) % n for i in range(n)]
    kv = [m.held[s] + 1 for s in src]
    gpu.inputs([1] * n, kv, src, m.held)
    before = _state(gpu)
    gpu.n_copies.fill_(9)
    with withheld():
        assert gpu.step() == fl.ERR_TIMEOUT == fl.flamia_get_device_status(gpu.pages_ws)
    assert all(torch.equal(a, b) for a, b in zip(_state(gpu), before)) and int(gpu.n_copies) == 0
    assert (gpu.slots == -1).all()
    copies = m.step([1] * n, kv, src)
    assert gpu.step() == fl.OK
    gpu.same(copies)
    assert gpu.slots.tolist() == m.slots([1] * n, kv, 64 * n)
