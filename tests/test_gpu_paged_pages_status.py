"""PagedCall with shared pages says on the device what became of its page calls."""
import pytest
import torch

import precision_causal_attention_token_gb300 as fl

I32 = dict(dtype=torch.int32)


def _call(device, **kw):
    return fl.PagedCall(3, 24, 4, 2, 64, 16, 12, 4, layers=2, shared=True, device=device, **kw)


def test_status_words_lie_at_the_workspaces_heads():
    c = _call("cpu")
    for word, ws in ((c.status, c.ws), (c.pages_status, c.pages_ws)):
        assert word.shape == (1,) and word.dtype == torch.int32 and word.data_ptr() == ws.data_ptr() and int(word) == fl.OK


@pytest.mark.gpu
def test_a_refused_compaction_is_seen():
    c = _call("cuda")
    dev = dict(device="cuda", **I32)
    c.plan(torch.tensor([0, 20, 23, 23], **dev), torch.tensor([20, 3, 0], **dev))
    c.plan(torch.tensor([0, 0, 1, 1], **dev), torch.tensor([0, 4, 0], **dev))
    assert int(c.status) == int(c.pages_status) == fl.OK
    state = (c.block_table, c.refs, c.free_pages, c.n_free, c.k)
    before = [x.clone() for x in state]
    held, c.free_pages[0] = int(c.free_pages[0]), 99
    c.compact()
    assert int(c.pages_status) == fl.ERR_BAD_PAGE and int(c.status) == fl.OK
    c.free_pages[0] = held
    assert all(torch.equal(a, b) for a, b in zip(state, before))
    c.compact()
    assert int(c.pages_status) == fl.OK and int(c.n_free) == 11 and int(c.block_table[1, 0]) == 0


@pytest.mark.gpu
def test_a_refused_step_and_a_copy_out_of_range_are_seen():
    c = _call("cuda")
    dev = dict(device="cuda", **I32)
    c.plan(torch.tensor([0, 20, 23, 23], **dev), torch.tensor([20, 3, 0], **dev))
    c.plan(torch.tensor([0, 1, 2, 2], **dev), torch.tensor([65, 4, 0], **dev))  # more than a request's four pages
    assert int(c.status) == int(c.pages_status) == fl.ERR_BAD_SEQLENS
    c.plan(torch.tensor([0, 1, 2, 2], **dev), torch.tensor([21, 4, 0], **dev))
    assert int(c.status) == int(c.pages_status) == fl.OK
    fl.flamia_paged_copy(c.prob, c.caches, c.caches, torch.tensor([[0, 12]], **dev), torch.tensor([1], **dev), c.pages_ws)
    assert int(c.status) == fl.OK and int(c.pages_status) == fl.ERR_BAD_PAGE
