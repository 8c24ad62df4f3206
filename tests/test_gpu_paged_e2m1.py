"""The 4-bit cache on the GPU: appended rows against the definition, attention of every kernel against 64 bits."""
import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged4_ref import Step4, packed, quantize4, unpacked, values4

pytestmark = pytest.mark.gpu


def _same_rows(got, want, what):
    """Bytes equal, but for the sign of a zero code."""
    g, w = unpacked(got.cpu()), unpacked(want)
    assert torch.equal(torch.where(g == 8, 0, g), torch.where(w == 8, 0, w)), what


def _append(x, d, dtype, ps=16, pad=3, dev="cuda"):
    """Rows x [T, Hkv, d] as K (and twice that as V) appended to shuffled pages; codes, blocks, scales of the rows."""
    T, Hkv = x.shape[:2]
    pages = -(-T // ps)
    ids = torch.randperm(pages + 2, generator=torch.Generator().manual_seed(T))[:pages]
    i32 = dict(dtype=torch.int32, device=dev)
    cu, kv, table = torch.tensor([0, T], **i32), torch.tensor([T], **i32), ids.to(**i32)[None].contiguous()
    prob = fl.make_paged(T + pad, Hkv, Hkv, d, cu, kv, table, page_size=ps, n_pages=pages + 2,
                         cache_dtype=fl.E2M1, in_dtype=fl.F32 if dtype == torch.float32 else fl.BF16)
    ws = torch.full((fl.flamia_paged_workspace_size(prob),), 0x5A, dtype=torch.uint8, device=dev)
    slots = torch.full((T + pad,), 7, **i32)
    fl.flamia_paged_plan(prob, ws, slots)
    pool = (pages + 2, Hkv, ps)
    k, v = (torch.full((*pool, d // 2), 0xEE, dtype=torch.uint8, device=dev) for _ in range(2))
    kb, vb = (torch.full((*pool, d // 16), 0xEE, dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.full(pool, 0xEE, dtype=torch.uint8, device=dev) for _ in range(2))
    rows = torch.full((T + pad, Hkv, d), float("nan"), dtype=dtype, device=dev)
    rows[:T] = x.to(dev, dtype)
    fl.flamia_paged_append(prob, rows, rows * 2, slots, fl.paged_cache(k, v, ks, vs, kb, vb), ws)
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(ws) == fl.OK
    t = torch.arange(T)
    page, off = ids[t // ps].to(dev), (t % ps).to(dev)
    untouched = torch.ones(pages + 2, ps, dtype=torch.bool, device=dev)
    untouched[page, off] = False
    for a in (k, v, kb, vb, ks, vs):
        assert (a.transpose(1, 2)[untouched] == 0xEE).all()
    at = lambda a: a[page, :, off]  # noqa: E731
    return [(at(k), at(kb), at(ks)), (at(v), at(vb), at(vs))], [rows[:T].cpu(), (rows[:T] * 2).cpu()]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,Hkv,ps,T", [(64, 1, 16, 1), (128, 3, 32, 33), (128, 8, 64, 200), (64, 5, 128, 517)])
def test_appended_rows_are_the_definitions(dtype, d, Hkv, ps, T):
    g = torch.Generator().manual_seed(d + T)
    x = torch.randn(T, Hkv, d, generator=g) * torch.exp(0.5 * torch.randn(T, Hkv, 1, generator=g))
    x[..., ::37] *= 6.0
    got, rows = _append(x, d, dtype, ps)
    for (c, b, s), r in zip(got, rows):
        wc, wb, ws = quantize4(r)
        assert torch.equal(s.cpu(), ws) and torch.equal(b.cpu(), wb)
        _same_rows(c, packed(wc), "codes")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_appended_rows_at_borders(dtype):
    """Every border between two codes and its neighbours under every block scale; sizes from subnormal to the largest."""
    d, rows = 128, []
    tie = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
    for code in range(1, 127):
        s = torch.tensor([code], dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        row = torch.zeros(8, 16, dtype=torch.float64)
        row[0, 0] = 2688.0  # exponent 0
        for i, f in enumerate((1.0, 1 + step, 1 - step, 1 + 2 * step, -1.0, -1 - step)):
            row[1 + i, :7] = tie * s * f
            row[1 + i, 15] = 6 * s
        rows.append(row.flatten())
    x = torch.stack(rows).to(dtype).double()
    # the same at other exponents; zeros; single values; what is not finite
    x = torch.cat([x, x * 2.0 ** -126, x * 2.0 ** 100, x * 2.0 ** -140])
    odd = torch.zeros(9, d, dtype=torch.float64)
    odd[1, 5], odd[2, 5], odd[3, 5] = 2.0 ** -133, -3.0e38, 1.0
    odd[4, 7], odd[5, 7], odd[6, 7] = float("inf"), float("nan"), -float("inf")
    odd[7] = -0.0
    odd[8, :64] = 2.0 ** -20
    x = torch.cat([x, odd]).to(dtype)[:, None]
    x = torch.cat([x, x.flip(0)], 1)
    got, rows = _append(x, d, dtype, 64)
    for (c, b, s), r in zip(got[:1], rows[:1]):
        wc, wb, ws = quantize4(r)
        assert torch.equal(s.cpu(), ws) and torch.equal(b.cpu(), wb)
        _same_rows(c, packed(wc), "codes")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,Hkv", [(64, 3), (128, 5), (64, 9)])
def test_append_from_a_fused_projection_into_chosen_slots(dtype, d, Hkv):
    """Rows at a stride, K and V of one buffer; slots in any order, skipped ones, one outside the pool (reported)."""
    T, ps, n, i32 = 45, 32, 7, dict(dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(d)
    width = (4 * Hkv + 2 * Hkv) * d
    rows = torch.randn(T, width, generator=g).to(dtype).cuda()
    k, v = rows[:, 4 * Hkv * d:5 * Hkv * d], rows[:, 5 * Hkv * d:]
    cu, kv, table = torch.tensor([0, T], **i32), torch.tensor([T], **i32), torch.zeros(1, 4, **i32)
    prob = fl.make_paged(T, 4 * Hkv, Hkv, d, cu, kv, table, page_size=ps, n_pages=n, cache_dtype=fl.E2M1, kv_stride=width,
                         in_dtype=fl.F32 if dtype == torch.float32 else fl.BF16)
    ws = torch.zeros(fl.flamia_paged_workspace_size(prob), dtype=torch.uint8, device="cuda")
    fl.flamia_paged_plan(prob, ws)
    slots = torch.randperm(n * ps, generator=g)[:T].int()
    slots[::7] = -1
    bad = slots.clone()
    bad[10], bad[11] = n * ps, -2
    pools = [torch.full((n, Hkv, ps, w), 0xEE, dtype=torch.uint8, device="cuda") for w in (d // 2, d // 2, 1, 1, d // 16, d // 16)]
    cache = fl.paged_cache(pools[0], pools[1], pools[2][..., 0], pools[3][..., 0], pools[4], pools[5])
    for s, status in ((slots, fl.OK), (bad, fl.ERR_BAD_PAGE)):
        for x in pools:
            x.fill_(0xEE)
        fl.flamia_paged_append(prob, k, v, s.cuda(), cache, ws)
        assert fl.flamia_get_device_status(ws) == status
        for x, (c, b, e) in ((k, (0, 4, 2)), (v, (1, 5, 3))):
            wc, wb, we = quantize4(x.reshape(T, Hkv, d).cpu())
            flat = [pools[i].transpose(1, 2).reshape(n * ps, Hkv, -1).cpu() for i in (c, b, e)]
            live = (s >= 0) & (s < n * ps)
            at = s[live].long()
            _same_rows(flat[0][at], packed(wc)[live], "codes")
            assert torch.equal(flat[1][at], wb[live]) and torch.equal(flat[2][at][..., 0], we[live])
            rest = torch.ones(n * ps, dtype=torch.bool)
            rest[at] = False
            assert all((y[rest] == 0xEE).all() for y in flat)


LENS = {  # (new tokens, cached after them)
    "one": ([1], [1]), "first": ([1, 1, 1], [1, 16, 17]), "decode": ([1] * 7, [3, 64, 65, 200, 1000, 1, 257]),
    "idle": ([1, 0, 1, 1], [0, 40, 33, 0]), "long": ([1], [9000]), "many": ([1] * 40, [37 * i % 300 + 1 for i in range(40)])}


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,Hkv,d,ps", [(4, 4, 64, 16), (8, 2, 128, 16), (8, 1, 128, 64), (15, 3, 64, 128), (12, 1, 128, 32), (40, 2, 64, 32)])
def test_single_tokens(lens, H, Hkv, d, ps):
    Step4(*LENS[lens], H=H, Hkv=Hkv, d=d, ps=ps, max_q=1, pad=2, poison=True, seed=len(lens)).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hkv,d,ps,max_q", [(4, 2, 128, 16, 4), (4, 2, 64, 64, 4), (4, 1, 128, 32, 4), (4, 1, 64, 16, 4), (4, 1, 128, 128, 8),
                                              (4, 1, 64, 16, 8), (6, 2, 128, 16, 8)])
def test_drafted_tokens(causal, H, Hkv, d, ps, max_q):
    q = [max_q, 1, 2, 0, max_q - 1, 3]
    Step4(q, [max_q, 90, 1, 50, 700, 258], H=H, Hkv=Hkv, d=d, ps=ps, max_q=max_q, causal=causal, pad=1, poison=True).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hkv,d,ps", [(2, 1, 128, 16), (4, 4, 64, 32), (10, 2, 128, 64), (3, 1, 64, 128), (12, 1, 128, 32), (34, 2, 64, 16)])
@pytest.mark.parametrize("q,kv", [([300], [300]), ([129, 1, 70], [500, 333, 70]), ([64, 200, 5, 1], [1000, 210, 3, 0]), ([257, 33], [2000, 40])])
def test_chunks_and_mixed(causal, H, Hkv, d, ps, q, kv):
    Step4(q, kv, H=H, Hkv=Hkv, d=d, ps=ps, causal=causal, pad=5, poison=True, seed=sum(q)).check()


@pytest.mark.parametrize("q,max_q", [([1, 1], 1), ([4, 3], 4), ([8, 5], 8), ([200, 150], 0)])
def test_strided_pools_and_queries(q, max_q):
    Step4(q, [300, 420], H=8, Hkv=2, d=128, ps=16, max_q=max_q, strided=True, q_extra=64).check()
    Step4(q, [300, 420], H=4, Hkv=2, d=64, ps=64, max_q=max_q, strided=True, scale=0.3).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,q,max_q", [(4, [1, 1], 1), (4, [3, 4], 4), (4, [8, 6], 8), (2, [100, 80], 0)])
def test_rows_of_very_different_size(d, H, q, max_q):
    """V rows up to 2^40 apart: f16 weights do not reach, the decode kernels take their careful pass."""
    for span in (10, 40, 80):
        g = torch.Generator().manual_seed(span)
        Step4(q, [400, 555], H=H, Hkv=1, d=d, ps=32, max_q=max_q,
              shift=lambda *s: torch.randint(-span, span + 1, s, generator=g)).check()


@pytest.mark.parametrize("H,q,max_q", [(4, [1, 1], 1), (4, [8, 6], 8), (2, [200, 130], 0)])
def test_large_rows(H, q, max_q):
    """Exponent bytes above 134: two factors in the tiles' conversion."""
    Step4(q, [400, 555], H=H, Hkv=1, d=128, ps=32, max_q=max_q, shift=lambda *s: torch.full(s, 30)).check()


@pytest.mark.parametrize("k_shift", [-112, -60, -14, -6, 5, 9, 40, 113])
@pytest.mark.parametrize("H,q,max_q", [(4, [1, 1], 1), (4, [8, 6], 8), (2, [200, 130], 0)])
def test_keys_and_queries_of_extreme_size(k_shift, H, q, max_q):
    """Scores of the usual size from keys times 2^k and queries times 2^-k: K's tiles with and without their exponents."""
    Step4(q, [400, 555], H=H, Hkv=1, d=128, ps=32, max_q=max_q, k_shift=k_shift, poison=True).check()


@pytest.mark.parametrize("low,high", [(-6, 6), (-7, 6), (-9, 9), (8, 12), (-16, -9)])
def test_tiles_at_the_border_of_f16(low, high):
    """Exponents that a tile of f16 holds (bytes 112 to 127), and some that it does not, block by block."""
    g = torch.Generator().manual_seed(low)

    def shift(n, h, ps):
        s = torch.randint(low, high + 1, (n, h, ps), generator=g)
        s[n // 2:] = 0  # some blocks are usual
        return s

    Step4([300, 77], [900, 431], H=4, Hkv=2, d=128, ps=128, shift=shift, poison=True).check()
    Step4([300, 77], [900, 431], H=2, Hkv=2, d=64, ps=16, shift=shift).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,q,max_q", [(4, 4, 4), (4, 8, 8), (2, 200, 0)])
def test_a_row_that_is_not_finite_stays_with_those_that_see_it(d, H, q, max_q):
    """V (then K) of the last token but two is NaN: rows before it do not change, the others are NaN (V: O only).

    The exponent that the f16 weights are relative to may change with the row, so O is compared as two roundings of one
    value: each half a bf16 step of it and f16's 2^-12 of the summed magnitudes off (2^-9 in the tile kernel, the same
    in both).  A block with such a row sums its weights in another order: two fp32 sums of up to 277 positive terms
    differ by at most 2 * 277 * 2^-24 of the sum, lse so by 2^-14.8 and twice half a step of values below 16 (2^-21)."""
    s = Step4([q], [q + 77], H=H, Hkv=1, d=d, ps=16, max_q=max_q)
    j = q + 77 - 3
    page, off = s.table_host[0][j // 16], j % 16
    O0, lse0 = (x.clone() for x in s.run())
    tol = 1.01 * (2.0 ** -8 * O0.double().abs() + 2.0 ** -11 * float(s.rows_of(0, 0)[1].abs().max()))[:q - 3]
    s.vs[page, 0, off] = 255
    s.v[page, 0, off], s.vb[page, 0, off] = 0xFF, 0x7F
    O, lse = s.run()
    assert fl.flamia_get_device_status(s.ws) == fl.OK
    assert ((O.double() - O0.double())[:q - 3].abs() <= tol).all() and torch.isnan(O[q - 3:]).all()
    assert ((lse - lse0).abs() <= 2.0 ** -14).all()
    s.vs[page, 0, off], s.ks[page, 0, off] = 127, 255
    s.v[page, 0, off], s.vb[page, 0, off] = 0, 0
    O, lse = s.run()
    assert torch.isfinite(O[:q - 3].float()).all() and torch.isnan(O[q - 3:]).all() and torch.isnan(lse[:, q - 3:]).all()
    assert ((lse - lse0)[:, :q - 3].abs() <= 2.0 ** -14).all()


def test_captured_and_replayed_equals_eager():
    for q, max_q in (([1, 1, 1], 1), ([130, 1, 20], 0)):
        s = Step4(q, [900, 31, 20], H=8, Hkv=2, d=128, max_q=max_q)
        O, lse = (x.clone() for x in s.run())
        g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            O2, lse2 = s.run()
        for _ in range(3):
            O2.fill_(5.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(O, O2) and torch.equal(lse, lse2)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes of codes, and more than 2^32 values before them; pages at its far end."""
    Hkv, ps, d, n = 8, 128, 128, 70000
    s = Step4([1, 60], [300, 200], H=8, Hkv=Hkv, d=d, ps=ps)
    far = torch.arange(n - s.n_pages, n)
    new = [torch.zeros(n, *x.shape[1:], dtype=torch.uint8, device="cuda") for x in (s.k, s.v, s.ks, s.vs, s.kb, s.vb)]
    for a, b in zip(new, (s.k, s.v, s.ks, s.vs, s.kb, s.vb)):
        a[far.cuda()] = b
    want, lse = (x.clone() for x in s.run())
    s.table.add_(n - s.n_pages)
    s.prob.n_pages = n
    s.pool = fl.paged_cache(*new)
    O, l2 = s.run()
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(s.ws) == fl.OK
    assert torch.equal(O, want) and torch.equal(lse, l2)


def test_serving_steps():
    """PagedCall over a 4-bit cache: a prompt, tokens one by one, drafts; each step against the rows that were given."""
    T, H, Hkv, d, ps = 300, 8, 2, 128, 32
    pc = fl.PagedCall(n_req=3, T=T, H=H, Hkv=Hkv, d=d, page_size=ps, n_pages=60, max_pages=40, layers=2, cache_dtype=fl.E2M1)
    g = torch.Generator(device="cuda").manual_seed(3)
    kv, held = [0, 0, 0], [[[], [], []] for _ in range(2)]
    for q in ([150, 33, 0], [1, 1, 90], [1, 1, 1], [6, 0, 3], [1, 200, 1]):
        kv = [a + b for a, b in zip(kv, q)]
        cu = torch.tensor([sum(q[:i]) for i in range(4)], dtype=torch.int32)
        pc.plan(cu.cuda(), torch.tensor(kv, dtype=torch.int32, device="cuda"))
        for layer in range(2):
            k, v = (torch.randn(T, Hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
            x = (2 * torch.randn(T, H, d, generator=g, device="cuda")).bfloat16()
            pc.append(layer, k, v)
            O, lse = pc.attend(layer, x)
            torch.cuda.synchronize()
            assert fl.flamia_get_device_status(pc.ws) == fl.OK
            for r in range(3):
                at = slice(int(cu[r]), int(cu[r + 1]))
                held[layer][r].append(tuple(values4(packed(c), b, s).cuda() for c, b, s in (quantize4(k[at].cpu()), quantize4(v[at].cpu()))))
                K, V = (torch.cat([h[i] for h in held[layer][r]]) for i in range(2))
                n = q[r]
                if not n:
                    continue
                assert K.shape[0] == kv[r]
                see = torch.arange(kv[r], device="cuda")[None] <= torch.arange(kv[r] - n, kv[r], device="cuda")[:, None]
                for h in range(H):
                    z = torch.where(see, x[at, h].double() @ K[:, h // 4].T / d ** 0.5, -torch.inf)
                    w = torch.softmax(z, 1)
                    # bf16 weights (2^-8) and result (2^-8), and 2^-13 for scores in fp32
                    tol = 2.0 ** -8 * (w @ V[:, h // 4]).abs() + (2.0 ** -8 + 2.0 ** -13) * 2 * (w @ V[:, h // 4].abs())
                    assert ((O[at, h].double() - w @ V[:, h // 4]).abs() <= tol).all()
                    assert ((lse[h, at].double() - torch.logsumexp(z, 1)).abs() <= 2.0 ** -12).all()
