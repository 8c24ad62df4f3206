"""The 4-bit cache without a GPU: refusals before any launch, and the tests' own model of its rows."""
import os
import re

import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged4_ref import packed, quantize4, unpacked, values4


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return fl.load_library()


def _prob(**kw):
    f = dict(n_req=3, T=6, max_q=4, H=4, Hkv=2, d=64, page_size=16, n_pages=8, max_pages=3, cache_dtype=fl.E2M1,
             in_dtype=fl.BF16, causal=1, softmax_scale=0.0, cu_q=0x10000, kv_len=0x20000, block_table=0x30000)
    f.update(kw)
    return fl.Paged(**f)


def test_problems_with_a_4_bit_cache_are_taken(lib):
    assert fl.flamia_paged_workspace_size(_prob()) == fl.flamia_paged_workspace_size(_prob(cache_dtype=fl.E4M3)) > 0
    assert fl.flamia_paged_workspace_size(_prob(cache_dtype=4)) == 0
    assert fl.flamia_paged_workspace_size(_prob(in_dtype=fl.E2M1)) == 0


@pytest.mark.parametrize("c", [
    dict(k_blocks=None), dict(v_blocks=None), dict(k_blocks=0x80008), dict(v_blocks=0x90004), dict(k_scales=None),
    dict(v_scales=0x70008), dict(page_stride=2 * 16 * 64 - 32), dict(page_stride=2 * 16 * 64 + 16), dict(k=None), dict(v=0x50008)])
def test_caches_are_checked(lib, c):
    f = dict(k=0x40000, v=0x50000, k_scales=0x60000, v_scales=0x70000, page_stride=0, k_blocks=0x80000, v_blocks=0x90000)
    f.update(c)
    cache, p, big = fl.Cache(**f), _prob(), 1 << 40
    assert lib.flamia_paged_append(p, 0x60000, 0x70000, 0x80000, cache, 0x100000, big, None) == fl.ERR_INVALID_ARG
    assert lib.flamia_paged_fwd(p, 0x60000, cache, 0x70000, None, 0x100000, big, None) == fl.ERR_INVALID_ARG


def test_binding_checks_the_pools(monkeypatch):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    k, sc, bl = u8(8, 2, 16, 32), u8(8, 2, 16), u8(8, 2, 16, 4)
    ok = fl.paged_cache(k, k.clone(), sc, sc, bl, bl)
    assert ok.pool == ((2, 16, 64, fl.E2M1), 8) and ok.page_stride == 2 * 16 * 64
    both = u8(8, 2, 2, 16, 32)
    assert fl.paged_cache(both[:, 0], both[:, 1], sc, sc, bl, bl).page_stride == 2 * 2 * 16 * 64
    fl.paged_cache(k, k, sc, sc, bl.view(torch.float8_e4m3fn), bl.view(torch.float8_e4m3fn))
    for args in ((k, k, sc, sc, bl, None), (k, k, sc, sc, None, bl), (k, k, sc, sc, bl[..., :3], bl[..., :3]),
                 (k, k, sc, sc, bl.int(), bl.int()), (k, k, None, None, bl, bl), (k, k, sc, None, bl, bl),
                 (k, k, sc, sc, bl[:7], bl[:7]), (k.view(torch.int8), k.view(torch.int8), sc, sc, bl, bl),
                 (k, k, sc, sc, bl.transpose(1, 2), bl.transpose(1, 2)), (k, k, sc, sc, u8(8, 2, 16, 8)[..., ::2], bl)):
        with pytest.raises(ValueError):
            fl.paged_cache(*args)
    monkeypatch.setattr(fl, "_paged_call", lambda *a: None)
    x = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    e4m3 = fl.paged_cache(u8(8, 2, 16, 64), u8(8, 2, 16, 64), sc, sc)
    for p, cache, fits in ((_prob(), ok, True), (_prob(cache_dtype=fl.E4M3), ok, False), (_prob(), e4m3, False),
                           (_prob(d=128), ok, False), (_prob(n_pages=9), ok, False), (_prob(page_size=32), ok, False)):
        for call in (lambda: fl.flamia_paged_append(p, x, x, x, cache, sc), lambda: fl.flamia_paged_fwd(p, x, cache, x, None, sc)):
            if fits:
                call()
            else:
                with pytest.raises(fl.FlamiaError):
                    call()


def test_model_of_the_rows():
    """By hand: 2688 is the largest value of exponent 0; a block's scale is the smallest that holds it; ties to even."""
    x = torch.zeros(5, 32)
    x[0, 0], x[0, 16] = 2688.0, 1.0        # e = 0, s = 448 and the first >= 1/6 = 0.171875
    x[1, 3] = -2689.0                      # e = 1, s: the first >= 224.083 = 240
    x[2, :9] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25])
    x[2, 16] = 2688.0
    x[4, 0] = float("inf")
    code, blocks, scales = quantize4(x)
    assert scales.tolist() == [127, 128, 127, 127, 255]
    b = blocks.view(torch.float8_e4m3fn).float()
    assert b[0].tolist() == [448.0, 0.171875] and b[1].tolist() == [240.0, 0.0] and b[2].tolist() == [1.0, 448.0]
    assert code[0, 0] == 7 and code[0, 16] == 7  # 1 / 0.171875 = 5.8 -> 6
    assert code[1, 3] == 8 + 7                   # 1344.5 / 240 = 5.6
    assert code[2, :9].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8]
    v = values4(packed(code), blocks, scales)
    assert torch.equal(unpacked(packed(code)), code)
    assert v[1, 3] == -2880.0 and v[2, :8].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    assert (v[3] == 0).all() and torch.isnan(v[4]).all()


def test_model_holds_every_row_within_a_step():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(500, 64, generator=g).double() * torch.exp2(torch.randint(-150, 120, (500, 1), generator=g).double())
    code, blocks, scales = quantize4(x.float())
    v = values4(packed(code), blocks, scales)
    s = torch.ldexp(blocks.view(torch.float8_e4m3fn).double(), (scales.int() - 127)[..., None]).repeat_interleave(16, -1)
    assert ((v - x.float().double()).abs() <= s).all()  # half the largest step, 2
    assert (v.abs() <= 6 * s).all()


@pytest.mark.parametrize("M,N,a_mn,b_mn", [(128, 128, 0, 0), (128, 128, 0, 1), (128, 64, 0, 1)])
def test_f16_instruction_descriptor(lib, M, N, a_mn, b_mn):
    """Bit fields of the kind::f16 instruction descriptor with f16 operands, each read back by itself."""
    x = fl.flamia_debug_mma_idesc(fl.MMA_F16, M, N, a_mn, b_mn)
    field = lambda lo, hi: (x >> lo) & ((1 << (hi - lo + 1)) - 1)  # noqa: E731
    assert field(0, 3) == 0 and field(6, 6) == 0 and field(13, 14) == 0
    assert field(4, 5) == 1  # fp32 accumulator
    assert field(7, 9) == 0 and field(10, 12) == 0  # f16, both operands
    assert (field(15, 15), field(16, 16)) == (a_mn, b_mn)
    assert field(17, 22) == N >> 3 and field(24, 28) == M >> 4 and field(23, 23) == 0 and field(29, 31) == 0
    assert x == fl.flamia_debug_mma_idesc(fl.MMA_BF16, M, N, a_mn, b_mn) & ~0x1F80
    with pytest.raises(fl.FlamiaError):
        fl.flamia_debug_mma_idesc(fl.MMA_F16, M, N, a_mn, b_mn, 1, 0)


def test_kernels_use_the_checked_f16_descriptors():
    src = open(os.path.join(os.path.dirname(fl.__file__), "csrc", "paged_chunk.cu")).read()
    assert set(re.findall(r"\bf16_idesc\([^()]*\)", src)) == {"f16_idesc(128, 128, 0, 0)", "f16_idesc(128, D, 0, 1)"}


def test_paged_call_holds_the_pools_of_each_type():
    for dt, width in ((fl.BF16, 64), (fl.E4M3, 64), (fl.E2M1, 32)):
        c = fl.PagedCall(n_req=2, T=6, H=4, Hkv=2, d=64, page_size=16, n_pages=8, max_pages=3, layers=3, device="cpu", cache_dtype=dt)
        assert c.k.shape == (3, 8, 2, 16, width) and len(c.caches) == 3
        assert all(x.pool == ((2, 16, 64, dt), 8) for x in c.caches)
        assert (c.k_blocks is None) == (dt != fl.E2M1) and (c.k_scales is None) == (dt == fl.BF16)
        assert c.caches[1].k == c.k[1].data_ptr()
