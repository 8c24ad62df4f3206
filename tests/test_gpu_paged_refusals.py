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
