"""A pool, its scales and the workspace are on one CUDA device: refused before any launch."""
import pytest
import torch

import precision_causal_attention_token_gb300 as fl


def _prob(**kw):
    f = dict(n_req=3, T=6, max_q=4, H=4, Hkv=2, d=64, page_size=16, n_pages=8, max_pages=3, cache_dtype=fl.E2M1,
             in_dtype=fl.BF16, causal=1, softmax_scale=0.0, cu_q=0x10000, kv_len=0x20000, block_table=0x30000)
    f.update(kw)
    return fl.Paged(**f)


def _pool(width, dtype=torch.uint8):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    k = torch.zeros(8, 2, 16, width, dtype=dtype)
    if dtype == torch.bfloat16:
        return [k, k.clone()]
    pool = [k, k.clone(), u8(8, 2, 16), u8(8, 2, 16)]
    return pool + [u8(8, 2, 16, 4), u8(8, 2, 16, 4)] if width == 32 else pool


@pytest.mark.parametrize("pool", [_pool(64, torch.bfloat16), _pool(64), _pool(32)])
def test_pools_over_two_devices_are_refused(pool):
    fl.paged_cache(*pool)
    fl.paged_cache(*[x.to("meta") for x in pool])
    for i in range(len(pool)):
        with pytest.raises(ValueError):
            fl.paged_cache(*[x.to("meta") if j == i else x for j, x in enumerate(pool)])


def test_a_pool_of_another_device_than_the_workspace_is_refused(monkeypatch):
    calls = []
    monkeypatch.setattr(fl, "_paged_call", lambda name, *a: calls.append(name))
    x, ws, cache = torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.zeros(16), fl.paged_cache(*_pool(32))
    here = cache.device
    for device in (here, 1):
        cache.device = device  # 1: as of a pool on another GPU
        for call in (lambda: fl.flamia_paged_append(_prob(), x, x, x, cache, ws), lambda: fl.flamia_paged_fwd(_prob(), x, cache, x, None, ws)):
            if device == here:
                call()
            else:
                with pytest.raises(fl.FlamiaError):
                    call()
    assert calls == ["flamia_paged_append", "flamia_paged_fwd"]


def test_a_workspace_in_host_memory_is_refused():
    """The kernels would be handed host addresses; with all arrays on the host the devices agree."""
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    ws, x, cache = torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(6, 4, 64, dtype=torch.bfloat16), fl.paged_cache(*_pool(32))
    p = _prob()
    for call in (lambda: fl.flamia_paged_plan(p, ws, i(6)), lambda: fl.flamia_paged_append(p, x, x, i(6), cache, ws),
                 lambda: fl.flamia_paged_fwd(p, x, cache, x, None, ws),
                 lambda: fl.flamia_paged_plan_shared(p, ws, ws, i(6), i(3), i(3), i(8), i(8), i(1), i(1), i(3, 2), i(1)),
                 lambda: fl.flamia_paged_copy(p, [cache], [cache], i(3, 2), i(1), ws),
                 lambda: fl.flamia_paged_compact(p, ws, i(3), i(8), i(8), i(1), i(8, 2), i(1))):
        with pytest.raises(fl.FlamiaError) as e:
            call()
        assert e.value.status == fl.ERR_INVALID_ARG
