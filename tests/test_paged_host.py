"""Host rules of the paged-cache entry points: refusals before any launch (no
pointer below is dereferenced), the workspace size, and the tests' own model."""
import os
import random
import re

import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged_ref import model_plan, pages_of, quantize_rows, row_values


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return fl.load_library()


def _prob(**kw):
    f = dict(n_req=3, T=40, max_q=4, H=8, Hkv=2, d=128, page_size=16, n_pages=100, max_pages=9, cache_dtype=fl.BF16,
             in_dtype=fl.BF16, causal=1, softmax_scale=0.0, cu_q=0x10000, kv_len=0x20000, block_table=0x30000)
    f.update(kw)
    return fl.Paged(**f)


BAD = [(dict(n_req=0), fl.ERR_INVALID_ARG), (dict(T=0), fl.ERR_INVALID_ARG), (dict(max_q=-1), fl.ERR_INVALID_ARG),
       (dict(max_q=41), fl.ERR_INVALID_ARG), (dict(H=9), fl.ERR_INVALID_ARG), (dict(Hkv=0), fl.ERR_INVALID_ARG),
       (dict(n_pages=0), fl.ERR_INVALID_ARG), (dict(max_pages=0), fl.ERR_INVALID_ARG),
       (dict(cu_q=None), fl.ERR_INVALID_ARG), (dict(kv_len=None), fl.ERR_INVALID_ARG),
       (dict(block_table=None), fl.ERR_INVALID_ARG), (dict(cu_q=0x10002), fl.ERR_INVALID_ARG),
       (dict(softmax_scale=-1.0), fl.ERR_INVALID_ARG), (dict(softmax_scale=float("nan")), fl.ERR_INVALID_ARG),
       (dict(softmax_scale=float("inf")), fl.ERR_INVALID_ARG), (dict(q_stride=1016), fl.ERR_INVALID_ARG),
       (dict(q_stride=1028), fl.ERR_INVALID_ARG), (dict(kv_stride=248), fl.ERR_INVALID_ARG),
       (dict(kv_stride=260), fl.ERR_INVALID_ARG), (dict(d=96), fl.ERR_UNSUPPORTED), (dict(page_size=8), fl.ERR_UNSUPPORTED),
       (dict(page_size=48), fl.ERR_UNSUPPORTED), (dict(page_size=256), fl.ERR_UNSUPPORTED),
       (dict(cache_dtype=fl.F32), fl.ERR_UNSUPPORTED), (dict(in_dtype=fl.E4M3), fl.ERR_UNSUPPORTED),
       (dict(n_req=8193), fl.ERR_UNSUPPORTED), (dict(H=258, Hkv=2), fl.ERR_UNSUPPORTED),
       (dict(n_pages=1 << 27), fl.ERR_UNSUPPORTED), (dict(max_pages=(1 << 26) + 1), fl.ERR_UNSUPPORTED),
       (dict(n_req=8192, max_pages=1 << 18), fl.ERR_UNSUPPORTED)]


@pytest.mark.parametrize("bad,want", BAD, ids=[str(b[0]) for b in BAD])
def test_bad_problems_are_refused(lib, bad, want):
    p, big, ws = _prob(**bad), 1 << 40, 0x100000
    c = fl.Cache(0x40000, 0x50000, None, None, 0)
    assert fl.flamia_paged_workspace_size(p) == 0
    assert lib.flamia_paged_plan(p, None, None, None, None, None, ws, big, None) == want
    assert lib.flamia_paged_append(p, 0x60000, 0x70000, 0x80000, c, ws, big, None) == want
    assert lib.flamia_paged_fwd(p, 0x60000, c, 0x70000, None, ws, big, None) == want


def test_null_problem_and_workspace(lib):
    assert fl.load_library().flamia_paged_workspace_size(None) == 0
    assert lib.flamia_paged_plan(None, None, None, None, None, None, 0x100000, 1 << 40, None) == fl.ERR_INVALID_ARG
    p = _prob()
    n = fl.flamia_paged_workspace_size(p)
    assert n > 0
    for ws, size, want in ((None, n, fl.ERR_INVALID_ARG), (0x100008, n, fl.ERR_INVALID_ARG),
                           (0x100000, n - 1, fl.ERR_WORKSPACE_TOO_SMALL)):
        assert lib.flamia_paged_plan(p, None, None, None, None, None, ws, size, None) == want


def test_page_management_takes_all_its_arrays_or_none(lib):
    p, args = _prob(), [0x40000, 0x50000, 0x60000, 0x70000]
    for i in range(4):
        some = list(args)
        some[i] = None
        assert lib.flamia_paged_plan(p, None, *some, 0x100000, 1 << 40, None) == fl.ERR_INVALID_ARG
        some[i] = args[i] + 1
        assert lib.flamia_paged_plan(p, None, *some, 0x100000, 1 << 40, None) == fl.ERR_INVALID_ARG
    assert lib.flamia_paged_plan(p, 0x80002, None, None, None, None, 0x100000, 1 << 40, None) == fl.ERR_INVALID_ARG


def test_caches_are_checked(lib):
    ws, big = 0x100000, 1 << 40
    e4 = dict(cache_dtype=fl.E4M3)
    cases = [({}, fl.Cache(None, 0x50000, None, None, 0)), ({}, fl.Cache(0x40000, None, None, None, 0)),
             ({}, fl.Cache(0x40008, 0x50000, None, None, 0)), ({}, fl.Cache(0x40000, 0x50000, 0x60000, 0x70000, 0)),
             ({}, fl.Cache(0x40000, 0x50000, None, None, 2 * 16 * 128 - 8)),
             ({}, fl.Cache(0x40000, 0x50000, None, None, 2 * 16 * 128 + 4)),
             (e4, fl.Cache(0x40000, 0x50000, None, None, 0)), (e4, fl.Cache(0x40000, 0x50000, 0x60000, None, 0)),
             (e4, fl.Cache(0x40000, 0x50000, 0x60000, 0x70008, 0)),
             (e4, fl.Cache(0x40000, 0x50000, 0x60000, 0x70000, 2 * 16 * 128 + 8))]
    for kw, c in cases:
        p = _prob(**kw)
        assert lib.flamia_paged_append(p, 0x60000, 0x70000, 0x80000, c, ws, big, None) == fl.ERR_INVALID_ARG
        assert lib.flamia_paged_fwd(p, 0x60000, c, 0x70000, None, ws, big, None) == fl.ERR_INVALID_ARG
    p, c = _prob(), fl.Cache(0x40000, 0x50000, None, None, 0)
    for k, v, s in ((None, 16, 16), (16, None, 16), (16, 16, None), (24, 16, 16), (16, 24, 16), (16, 16, 18)):
        assert lib.flamia_paged_append(p, k, v, s, c, ws, big, None) == fl.ERR_INVALID_ARG
    for q, O, lse in ((None, 16, 16), (16, None, 16), (24, 16, 16), (16, 24, 16), (16, 16, 18)):
        assert lib.flamia_paged_fwd(p, q, c, O, lse, ws, big, None) == fl.ERR_INVALID_ARG


def test_binding_checks_tensors():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    ok = dict(page_size=16, n_pages=4)
    fl.make_paged(4, 2, 1, 64, i32(3), i32(2), i32(2, 5), **ok)
    for cu, kv, tab in ((i32(2), i32(2), i32(2, 5)), (i32(3), i32(2), i32(3, 5)), (i32(3), i32(2), i32(10)),
                        (i32(3).long(), i32(2), i32(2, 5)), (i32(3), i32(2).float(), i32(2, 5)),
                        (i32(3), i32(2), i32(5, 2).t())):
        with pytest.raises(ValueError):
            fl.make_paged(4, 2, 1, 64, cu, kv, tab, **ok)
    k = torch.zeros(4, 2, 16, 64)
    fl.paged_cache(k, k)
    sc = torch.zeros(4, 2, 16, dtype=torch.uint8)
    both = torch.zeros(4, 2, 2, 16, 64)
    assert fl.paged_cache(both[:, 0], both[:, 1]).page_stride == 2 * 2 * 16 * 64
    for args in ((k, k[:2]), (k, k.half()), (k.transpose(1, 2), k.transpose(1, 2)), (k[0], k[0]),
                 (k, k, sc[:2], sc), (k, k, sc.int(), sc), (k, k, sc, sc.transpose(1, 2))):
        with pytest.raises(ValueError):
            fl.paged_cache(*args)


def test_status_strings_of_the_paged_conditions(lib):
    assert "pages" in fl.status_string(fl.ERR_NO_PAGES) and "page" in fl.status_string(fl.ERR_BAD_PAGE)


def test_model_of_the_pages():
    """The list model by hand: request 0 gives back two pages, request 1 takes three."""
    table, free, slots = model_plan([[4, 2, 9, -1], [7, -1, -1, -1]], [5, 3], [40, 10], [16, 50], [0, 40], 16, 43)
    # stack 5 3 2 9 -> request 1 takes 9, 2, 3
    assert table == [[4, 2, 9, -1], [7, 9, 2, 3]] and free == [5]
    assert slots[:7] == [7 * 16 + 10 + i for i in range(6)] + [9 * 16] and slots[-4:] == [3 * 16 + 1, -1, -1, -1]


def test_model_of_the_quantizer():
    x = torch.tensor([[448.0] * 4, [449.0, 1.0, 0.0, -2.0], [0.0] * 4, [2.0 ** -130] * 4])
    codes, sc = quantize_rows(x)
    assert sc.tolist() == [127, 128, 127, 0]
    assert row_values(codes, sc)[0].tolist() == [448.0] * 4
    assert row_values(codes, sc)[1].tolist() == [448.0, 1.0, 0.0, -2.0]  # 224.5 rounds to 224
    assert row_values(codes, sc)[3].tolist() == [2.0 ** -130] * 4
    r = random.Random(0)
    for _ in range(50):
        n, ps = r.randrange(0, 500), r.choice([16, 32])
        assert pages_of(n, ps) == (n + ps - 1) // ps


@pytest.mark.parametrize("M,N,a_mn,b_mn", [(128, 128, 0, 0), (128, 128, 0, 1), (128, 64, 0, 1), (64, 8, 1, 0)])
def test_bf16_instruction_descriptor(lib, M, N, a_mn, b_mn):
    """Bit fields of the kind::f16 instruction descriptor, each read back by itself."""
    x = fl.flamia_debug_mma_idesc(fl.MMA_BF16, M, N, a_mn, b_mn)
    field = lambda lo, hi: (x >> lo) & ((1 << (hi - lo + 1)) - 1)  # noqa: E731
    assert field(0, 3) == 0 and field(6, 6) == 0  # dense, no saturation
    assert field(4, 5) == 1  # fp32 accumulator
    assert field(7, 9) == 1 and field(10, 12) == 1  # bf16
    assert field(13, 14) == 0  # no negation
    assert (field(15, 15), field(16, 16)) == (a_mn, b_mn)
    assert field(17, 22) == N >> 3 and field(24, 28) == M >> 4 and field(23, 23) == 0 and field(29, 31) == 0


def test_bf16_instruction_descriptor_refusals(lib):
    for args in ((96, 128), (128, 120), (128, 128, 2, 0), (128, 128, 0, 0, 1, 0)):
        with pytest.raises(fl.FlamiaError):
            fl.flamia_debug_mma_idesc(fl.MMA_BF16, *args)


def test_kernels_use_the_checked_bf16_descriptors():
    src = open(os.path.join(os.path.dirname(fl.__file__), "csrc", "paged_chunk.cu")).read()
    assert set(re.findall(r"\bbf16_idesc\([^()]*\)", src)) == {"bf16_idesc(128, 128, 0, 0)", "bf16_idesc(128, D, 0, 1)"}


def test_a_chunk_call_holds_up_to_2_25_keys_a_request(lib):
    """The limit counts where some request may take the chunk kernel: more than 32 rows (here max_q * 4)."""
    for max_q, pages, ok in ((9, 1 << 21, True), (9, (1 << 21) + 1, False), (8, (1 << 21) + 1, True),
                             (8, 1 << 26, True), (0, (1 << 21) + 1, False)):
        p = _prob(max_q=max_q, max_pages=pages)
        assert (fl.flamia_paged_workspace_size(p) > 0) == ok
        if not ok:
            assert lib.flamia_paged_plan(p, None, None, None, None, None, 0x100000, 1 << 40, None) == fl.ERR_UNSUPPORTED


def test_paged_call_checks_what_it_is_given():
    """Shapes, dtypes and strides, before anything runs (tensors of T rows, whatever cu_q says)."""
    import torch
    c = fl.PagedCall(n_req=2, T=6, H=4, Hkv=2, d=64, page_size=16, n_pages=8, max_pages=3, device="cpu")
    kv, q = torch.zeros(6, 2, 64, dtype=torch.bfloat16), torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    cu, n = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    wide = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: c.append(0, kv[:5], kv), lambda: c.append(0, kv, kv[:5]), lambda: c.append(0, kv.float(), kv),
                 lambda: c.append(0, wide[:, :2], kv), lambda: c.attend(0, q[:5]), lambda: c.attend(0, q.half()),
                 lambda: c.attend(0, torch.cat([q, q], 1)[:, :4]), lambda: c.plan(cu[:2], n), lambda: c.plan(cu, n[:1]),
                 lambda: c.plan(cu.long(), n), lambda: c.plan(cu, n.long())):
        with pytest.raises(fl.FlamiaError) as e:
            call()
        assert e.value.status == fl.ERR_INVALID_ARG
