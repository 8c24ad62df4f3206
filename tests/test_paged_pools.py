"""What the Python entry points of the paged operators refuse of tensors, before anything is launched."""
import pytest
import torch

import precision_causal_attention_token_gb300 as fl


def _prob(**kw):
    f = dict(n_req=3, T=6, max_q=4, H=4, Hkv=2, d=64, page_size=16, n_pages=8, max_pages=3, cache_dtype=fl.BF16,
             in_dtype=fl.BF16, causal=1, softmax_scale=0.0, cu_q=0x10000, kv_len=0x20000, block_table=0x30000)
    f.update(kw)
    return fl.Paged(**f)


@pytest.mark.parametrize("pages,ok", [(8, True), (9, True), (7, False)])
def test_pools_of_too_few_pages_are_refused(pages, ok, monkeypatch):
    _refuses(_prob(), torch.zeros(pages, 2, 16, 64, dtype=torch.bfloat16), ok, monkeypatch)


@pytest.mark.parametrize("shape,dtype,cache_dtype,ok", [
    ((8, 2, 16, 64), torch.bfloat16, fl.BF16, True), ((8, 2, 16, 64), torch.float32, fl.BF16, False),
    ((8, 2, 16, 64), torch.float16, fl.BF16, False), ((8, 2, 16, 64), torch.uint8, fl.BF16, False),
    ((8, 2, 16, 64), torch.uint8, fl.E4M3, True), ((8, 2, 16, 64), torch.float8_e4m3fn, fl.E4M3, True),
    ((8, 2, 16, 64), torch.bfloat16, fl.E4M3, False), ((8, 2, 32, 64), torch.bfloat16, fl.BF16, False),
    ((8, 1, 16, 64), torch.bfloat16, fl.BF16, False), ((8, 2, 16, 128), torch.bfloat16, fl.BF16, False)])
def test_pools_of_another_kind_are_refused(shape, dtype, cache_dtype, ok, monkeypatch):
    _refuses(_prob(cache_dtype=cache_dtype), torch.zeros(shape, dtype=dtype), ok, monkeypatch)


def _refuses(prob, k, ok, monkeypatch):
    calls = []
    monkeypatch.setattr(fl, "_paged_call", lambda name, *args: calls.append(name))
    sc = [torch.zeros(k.shape[:3], dtype=torch.uint8)] * 2 if k.element_size() == 1 else []
    cache, x, ws = fl.paged_cache(k, k.clone(), *sc), torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.zeros(16)
    for call in (lambda: fl.flamia_paged_append(prob, x, x, x, cache, ws),
                 lambda: fl.flamia_paged_fwd(prob, x, cache, x, None, ws)):
        if ok:
            call()
        else:
            with pytest.raises(fl.FlamiaError) as e:
                call()
            assert e.value.status == fl.ERR_INVALID_ARG
    assert len(calls) == (2 if ok else 0)


def test_pages_that_share_memory_are_refused():
    """An expanded pool: one page's memory for all of them, which would be read and written as if it were a whole pool."""
    one, two = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(5 * 1024 + 2048, dtype=torch.bfloat16)
    fl.paged_cache(one, one)
    for k in (one.expand(4, -1, -1, -1), two.as_strided((5, 2, 16, 64), (1024, 1024, 64, 1))):
        with pytest.raises(ValueError):
            fl.paged_cache(k, k)


def test_paged_call_refuses_tensors_of_another_device():
    """Before anything is launched: a pointer of another device is no address on this one."""
    c = fl.PagedCall(n_req=2, T=6, H=4, Hkv=2, d=64, page_size=16, n_pages=8, max_pages=3, device="cpu")
    away = lambda h: torch.zeros(6, h, 64, dtype=torch.bfloat16, device="meta")  # noqa: E731
    here = torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: c.append(0, away(2), here), lambda: c.append(0, here, away(2)), lambda: c.attend(0, away(4))):
        with pytest.raises(fl.FlamiaError) as e:
            call()
        assert e.value.status == fl.ERR_INVALID_ARG
