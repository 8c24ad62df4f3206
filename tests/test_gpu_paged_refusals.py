"""Calls that the paged operators refuse on the device: the status word says so and nothing has been written."""
import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged_ref import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("q,H", [([1, 1], 2), ([20, 30], 2), ([2, 3], 17), ([2, 3], 32), ([2, 1], 128)])
def test_forward_alone_on_a_workspace_without_its_plan(cache, q, H):
    """Never planned (zeros), or planned for another problem that had no work: heads of every group size."""
    s = Step(q, [50, 60], H=H, Hkv=1, cache=cache, d=64, max_q=max(q))
    O, lse = torch.full((s.T, H, 64), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((H, s.T), 5.0, device="cuda")
    none = torch.zeros_like(s.cu_q)
    other = fl.make_paged(s.T, H, 1, 64, none, s.kv, s.table, page_size=s.ps, n_pages=s.n_pages + 1,
                          max_q=max(q), cache_dtype=s.prob.cache_dtype)
    for prepare in (lambda: s.ws.zero_(), lambda: fl.flamia_paged_plan(other, s.ws)):
        prepare()
        assert fl.flamia_get_device_status(s.ws) == fl.OK
        fl.flamia_paged_fwd(s.prob, s.q, s.pool, O, lse, s.ws)
        torch.cuda.synchronize()
        assert fl.flamia_get_device_status(s.ws) == fl.ERR_INVALID_ARG
        assert (O == 5).all() and (lse == 5).all()


@pytest.mark.parametrize("n,q,H,Hkv,fits", [(1, 1 << 15, 128, 1, False), (1, 1 << 13, 128, 1, True),
                                            (4, 1 << 19, 128, 128, False), (1, 1 << 19, 128, 128, True)])
def test_a_step_too_large_for_the_work_split_moves_no_page(n, q, H, Hkv, fits):
    """Tiles of 256 rows (2 tokens of 128 heads, 256 of one) times blocks of 128 keys: 2^14 x 2^18 of one head, or 4 x
    2^11 x 2^18 of 128 heads, are too many; a quarter of each is not.  A smaller step on the same buffers follows."""
    ps, keys = 128, 1 << 25
    pages, held = keys // ps, (keys - q) // ps
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((n, pages), -9, **i32)
    table[:, :held] = torch.arange(n * held, **i32).view(n, held)
    free = torch.arange(n * held, n * pages, **i32)
    free = torch.cat([free, torch.full((n * pages - free.numel(),), -3, **i32)])
    n_free, old = torch.tensor([n * (pages - held)], **i32), torch.full((n,), keys - q, **i32)
    cu, new = torch.arange(n + 1, **i32) * q, torch.full((n,), keys, **i32)
    slots = torch.full((n * q,), -7, **i32)
    prob = fl.make_paged(n * q, H, Hkv, 64, cu, new, table, page_size=ps, n_pages=n * pages)
    ws = torch.zeros(fl.flamia_paged_workspace_size(prob), dtype=torch.uint8, device="cuda")
    before = table.clone(), free.clone(), n_free.clone()
    fl.flamia_paged_plan(prob, ws, slots, old, free, n_free, n_free)
    torch.cuda.synchronize()
    if fits:
        assert fl.flamia_get_device_status(ws) == fl.OK and int(n_free) == 0 and (slots >= 0).all()
        return
    assert fl.flamia_get_device_status(ws) == fl.ERR_UNSUPPORTED
    assert all(torch.equal(a, b) for a, b in zip((table, free, n_free), before)) and (slots == -1).all()
    cu.copy_(torch.arange(n + 1, **i32))
    new.copy_(old + 1)
    fl.flamia_paged_plan(prob, ws, slots, old, free, n_free, n_free)
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(ws) == fl.OK and int(n_free) == n * (pages - held) - n
    assert (slots[:n] >= 0).all() and (slots[n:] == -1).all()
