"""Pages that requests share, without a GPU: refusals before any launch, and the tests' own model by hand."""
import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged_pages_ref import Pool


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return fl.load_library()


def _prob(**kw):
    f = dict(n_req=3, T=6, max_q=4, H=4, Hkv=2, d=64, page_size=16, n_pages=8, max_pages=3, cache_dtype=fl.BF16,
             in_dtype=fl.BF16, causal=1, softmax_scale=0.0, cu_q=0x10000, kv_len=0x20000, block_table=0x30000)
    f.update(kw)
    return fl.Paged(**f)


BIG = 1 << 40


def _share(lib, p, over=(), pages=(0x200000, BIG), ws=(0x100000, BIG)):
    args = [0x40000, 0x50000, 0x60000, 0x70000, 0x80000, 0x90000, 0xA0000, 0xB0000, 0xC0000]
    for i, x in dict(over).items():
        args[i] = x
    return lib.flamia_paged_plan_shared(p, *args, *pages, *ws, None)


def test_shared_plan_refusals(lib):
    p = _prob()
    size = fl.flamia_paged_pages_workspace_size(p)
    assert size > 0 and fl.flamia_paged_pages_workspace_size(_prob(d=96)) == 0
    assert lib.flamia_paged_pages_workspace_size(None) == 0
    for i in range(2, 9):  # old_len and behind: all there, all aligned
        for x in (None, 0x40002):
            assert _share(lib, p, {i: x}) == fl.ERR_INVALID_ARG
    for i in range(2):  # slot_map, src: may be left out
        assert _share(lib, p, {i: 0x40001}) == fl.ERR_INVALID_ARG
    assert _share(lib, p, pages=(None, BIG)) == _share(lib, p, pages=(0x200008, BIG)) == fl.ERR_INVALID_ARG
    assert _share(lib, p, pages=(0x200000, size - 1)) == fl.ERR_WORKSPACE_TOO_SMALL
    assert _share(lib, p, ws=(None, BIG)) == fl.ERR_INVALID_ARG
    assert _share(lib, p, ws=(0x100000, fl.flamia_paged_workspace_size(p) - 1)) == fl.ERR_WORKSPACE_TOO_SMALL
    assert _share(lib, _prob(page_size=8)) == fl.ERR_UNSUPPORTED and _share(lib, None) == fl.ERR_INVALID_ARG
    # a step that flamia_paged_plan might refuse for its amount of attention: 2^19 tokens of 128 heads over 2^25 keys
    assert _share(lib, _prob(T=1 << 19, max_q=0, H=128, Hkv=1, max_pages=1 << 18, page_size=128, n_pages=1 << 20)) == fl.ERR_UNSUPPORTED


def test_compact_and_copy_refusals(lib):
    p, ws = _prob(), (0x200000, BIG)
    args = [0x40000, 0x50000, 0x60000, 0x70000, 0x80000, 0x90000]
    for i in (0, 2, 3, 4, 5):
        for x in (None, 0x40002):
            a = list(args)
            a[i] = x
            assert lib.flamia_paged_compact(p, *a, *ws, None) == fl.ERR_INVALID_ARG
    assert lib.flamia_paged_compact(p, 0x40000, 0x50001, *args[2:], *ws, None) == fl.ERR_INVALID_ARG
    assert lib.flamia_paged_compact(p, *args[:4], 0x80004, 0x90000, *ws, None) == fl.ERR_INVALID_ARG
    size = fl.flamia_paged_pages_workspace_size(p)
    assert lib.flamia_paged_compact(p, *args, 0x200000, size - 1, None) == fl.ERR_WORKSPACE_TOO_SMALL
    c = (fl.Cache * 2)(fl.Cache(0x40000, 0x50000, None, None, 0), fl.Cache(0x40000, 0x50000, None, None, 0))
    bad = (fl.Cache * 2)(fl.Cache(0x40000, 0x50000, None, None, 0), fl.Cache(0x40000, 0x50008, None, None, 0))
    ok = [2, c, c, 0x60000, 5, 0x70000]
    for i, x in ((0, 0), (0, -1), (1, None), (2, None), (1, bad), (2, bad), (3, None), (3, 0x60002), (4, -1), (5, None), (5, 0x70001)):
        a = list(ok)
        a[i] = x
        assert lib.flamia_paged_copy(p, *a, *ws, None) == fl.ERR_INVALID_ARG
    assert lib.flamia_paged_copy(p, *ok, 0x200008, BIG, None) == fl.ERR_INVALID_ARG
    assert lib.flamia_paged_copy(p, *ok, 0x200000, size - 1, None) == fl.ERR_WORKSPACE_TOO_SMALL
    for dt in (fl.E4M3, fl.E2M1):  # pools without their scales
        assert lib.flamia_paged_copy(_prob(cache_dtype=dt), *ok, *ws, None) == fl.ERR_INVALID_ARG


def test_binding_checks_the_arrays(monkeypatch):
    calls = []
    monkeypatch.setattr(fl, "_paged_call", lambda name, *a: calls.append(name))
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    p, ws = _prob(), torch.zeros(16)
    share = dict(slot_map=i(6), src=i(3), old_len=i(3), refs=i(8), free_pages=i(8), n_free=i(1), n_free_out=i(1), copies=i(3, 2), n_copies=i(1))
    fl.flamia_paged_plan_shared(p, ws, ws, **share)
    fl.flamia_paged_plan_shared(p, ws, ws, **{**share, "slot_map": None, "src": None})
    for k, x in (("slot_map", i(5)), ("src", i(2)), ("old_len", i(2)), ("refs", i(7)), ("free_pages", i(7)), ("n_free", i(0)), ("n_free_out", i(0)),
                 ("copies", i(2, 2)), ("n_copies", i(0)), ("refs", i(8).long()), ("copies", i(3, 4)[:, ::2])):
        with pytest.raises(fl.FlamiaError) as e:
            fl.flamia_paged_plan_shared(p, ws, ws, **{**share, k: x})
        assert e.value.status == fl.ERR_INVALID_ARG
    comp = dict(length=i(3), refs=i(8), free_pages=i(8), n_free=i(1), copies=i(8, 2), n_copies=i(1))
    fl.flamia_paged_compact(p, ws, **comp)
    fl.flamia_paged_compact(p, ws, **{**comp, "refs": None})
    for k, x in (("length", i(2)), ("refs", i(7)), ("free_pages", i(7)), ("n_free", i(0)), ("copies", i(7, 2)), ("n_copies", i(0))):
        with pytest.raises(fl.FlamiaError):
            fl.flamia_paged_compact(p, ws, **{**comp, k: x})
    pool = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    c, small = fl.paged_cache(pool, pool.clone()), fl.paged_cache(pool[:7], pool[:7])
    fl.flamia_paged_copy(p, [c, c], [c, c], i(3, 2), i(1), ws)
    away = fl.paged_cache(pool.to("meta"), pool.to("meta"))
    away.device = 1  # as of a pool on another GPU
    for src, dst in (([c], [c, c]), ([], []), ([c], [small]), ([small], [c]), ([away], [c]), ([c], [away])):
        with pytest.raises(fl.FlamiaError):
            fl.flamia_paged_copy(p, src, dst, i(3, 2), i(1), ws)

    class Away:  # a tensor of another GPU
        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return 1

    for k in share:
        with pytest.raises(fl.FlamiaError):
            fl.flamia_paged_plan_shared(p, ws, ws, **{**share, k: Away(share[k])})
    with pytest.raises(fl.FlamiaError):
        fl.flamia_paged_plan_shared(p, ws, Away(ws), **share)
    for k in comp:
        with pytest.raises(fl.FlamiaError):
            fl.flamia_paged_compact(p, ws, **{**comp, k: Away(comp[k])})
    assert calls == ["flamia_paged_plan_shared"] * 2 + ["flamia_paged_compact"] * 2 + ["flamia_paged_copy"]


def test_paged_call_refuses_forks_of_unshared_pages():
    kw = dict(n_req=2, T=6, H=4, Hkv=2, d=64, page_size=16, n_pages=8, max_pages=3, device="cpu")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    c = fl.PagedCall(**kw)
    for call in (lambda: c.plan(i(3), i(2), i(2)), c.compact):
        with pytest.raises(fl.FlamiaError):
            call()
    c = fl.PagedCall(shared=True, **kw)
    for src in (i(3), i(2).long()):
        with pytest.raises(fl.FlamiaError):
            c.plan(i(3), i(2), src)


def test_model_by_hand():
    """Two answers to one prompt of 20 tokens on pages of 16: both write into the second page, the first keeps it."""
    m = Pool(3, 8, 3, 16)
    assert m.step([20, 0, 0], [20, 0, 0], [0, 1, 2]) == [] and m.table[0][:2] == [7, 6] and m.free == [0, 1, 2, 3, 4, 5]
    assert m.step([1, 1, 0], [21, 21, 0], [0, 0, 2]) == [[6, 5]]
    assert m.table[0][:2] == [7, 6] and m.table[1][:2] == [7, 5] and m.refs == [0, 0, 0, 0, 0, 1, 1, 2]
    # the second goes on as two, the first ends: its own page is free, the prompt's first page is not
    assert m.step([0, 1, 1], [0, 22, 22], [-1, 1, 1]) == [[5, 6]]
    assert m.table[1][:2] == [7, 5] and m.table[2][:2] == [7, 6] and m.refs[7] == 2 and m.free == [0, 1, 2, 3, 4]
    assert m.compact() == [[5, 0], [6, 1], [7, 2]]
    assert m.table[1][:2] == [2, 0] and m.table[2][:2] == [2, 1] and m.free == [7, 6, 5, 4, 3]
