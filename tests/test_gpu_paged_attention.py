"""flamia_paged_fwd against plain attention in 64 bits over the same cache."""
import math

import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged_ref import Step

pytestmark = pytest.mark.gpu

CACHES = ["bf16", "e4m3"]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_decode_lengths(cache, d, ps):
    """One new token: lengths from one on, around the page, chunk and block edges."""
    kv = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 300, 1000]
    Step([1] * len(kv), kv, H=4, Hkv=2, d=d, ps=ps, cache=cache, seed=ps + d, max_q=1).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (8, 1), (12, 4), (5, 1), (16, 1), (28, 2), (11, 1)])
def test_decode_head_groups(cache, H, Hkv):
    Step([1, 1, 1], [70, 333, 5], H=H, Hkv=Hkv, cache=cache, seed=H, max_q=1).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
def test_decode_long_context_is_split(cache, d):
    """One request over many workers, whose partial results are joined."""
    Step([1], [20011], H=8, Hkv=2, d=d, ps=64, cache=cache, seed=3, max_q=1).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("H", [8, 16, 32])
def test_one_head_split_over_every_worker(cache, H):
    """One tile for the whole GPU: hundreds of partial results in one join, at 8, 16 and 32 rows."""
    Step([1], [180011], H=H, Hkv=1, ps=128, cache=cache, seed=H, max_q=1).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("causal", [True, False])
def test_drafted_tokens(cache, causal):
    """A few new tokens a request, the decode kernel's 16 rows full and not, rows without a key."""
    Step([4, 1, 3, 2, 4], [200, 1, 3, 1, 77], H=8, Hkv=2, cache=cache, causal=causal, seed=5, max_q=4).check()
    Step([2, 1, 2], [129, 64, 1], H=4, Hkv=1, d=64, cache=cache, causal=causal, seed=6, max_q=2).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_drafted_tokens_of_32_rows(cache, d, causal):
    """Up to 32 rows of a key/value head; a long context, split; few rows beside many."""
    Step([8, 5, 1, 8, 3], [2000, 33, 9000, 8, 2], H=8, Hkv=2, d=d, cache=cache, causal=causal, seed=15, max_q=8).check()
    Step([2, 1], [700, 65], H=16, Hkv=1, d=d, ps=64, cache=cache, causal=causal, seed=16, max_q=2).check()
    Step([1, 1], [100, 300], H=32, Hkv=1, d=d, ps=32, cache=cache, causal=causal, seed=17, max_q=1).check()
    Step([10, 7], [100, 300], H=3, Hkv=1, d=d, ps=32, cache=cache, causal=causal, seed=18, max_q=10).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_chunk_lengths(cache, d, causal):
    """Chunks of many sizes over contexts of many sizes, some rows without a key, one request without tokens."""
    q = [1, 17, 64, 65, 130, 300, 0, 33, 20]
    kv = [1, 17, 100, 65, 700, 300, 50, 5, 128]
    Step(q, kv, H=4, Hkv=2, d=d, ps=16, cache=cache, causal=causal, pad=5, seed=d).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (6, 2), (7, 1), (16, 2), (12, 1), (40, 1)])
def test_chunk_head_groups(cache, H, Hkv):
    """Query heads a key/value head: powers of two and not, more than a half tile's worth of heads."""
    Step([50, 1, 90], [60, 200, 140], H=H, Hkv=Hkv, d=128, ps=32, cache=cache, seed=H).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("H", [65, 127, 128])
def test_chunk_large_head_groups(cache, H):
    """One token a half tile."""
    Step([3, 1], [60, 200], H=H, Hkv=1, d=64, ps=32, cache=cache, seed=1).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_chunk_page_sizes(cache, ps):
    Step([100, 257, 5], [1000, 300, 129], H=2, Hkv=1, ps=ps, cache=cache, seed=ps).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_long_context_is_split(cache, d):
    """One tile's keys over many workers."""
    Step([40], [9000], H=8, Hkv=2, d=d, ps=64, cache=cache, seed=9).check()


@pytest.mark.parametrize("cache", CACHES)
def test_mixed_batch(cache):
    """Chunks, decoding requests, inactive slots and a padded tail in one call."""
    q = [1, 150, 1, 1, 64, 1, 1, 1, 0, 1]
    kv = [500, 150, 0, 77, 1024, 1, 2048, 640, 0, 129]
    Step(q, kv, H=8, Hkv=2, ps=64, cache=cache, pad=9, seed=2).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_no_keys_at_all(cache, kind):
    s = Step([1, 1] if kind == "decode" else [20, 30], [0, 0], cache=cache, max_q=1 if kind == "decode" else 0)
    O, lse = s.run()
    assert (O == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("kind", ["decode", "chunk"])
@pytest.mark.parametrize("fill", [math.nan, math.inf])
def test_stale_slots_are_not_read_as_values(cache, kind, fill):
    """Slots past a request's last token hold what an earlier owner left: NaN and infinities there change nothing."""
    q, kv = ([1, 1, 1], [1, 130, 77]) if kind == "decode" else ([30, 1, 140], [30, 130, 333])
    for ps in (16, 128):
        Step(q, kv, ps=ps, cache=cache, fill=fill, seed=4, max_q=1 if kind == "decode" else 0, pad=2).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_nan_reaches_only_rows_that_see_it(cache, kind):
    """A NaN key, or a NaN value, of one request makes its rows NaN and no other's."""
    for which in ("k", "v"):
        s = Step([1, 1] if kind == "decode" else [20, 30], [50, 60], cache=cache, seed=8,
                 max_q=1 if kind == "decode" else 0)
        page, off = s.table_host[0][1], 3  # token 19 of request 0
        if cache == "bf16":
            (s.k if which == "k" else s.v)[page, :, off, 5] = math.nan
        else:
            (s.ks if which == "k" else s.vs)[page, :, off] = 255
        O, lse = s.run()
        n = s.q_len[0]
        bad = torch.isnan(O[:n])
        assert bad[..., 5].all() if which == "v" and cache == "bf16" else bad.all()
        assert torch.isnan(lse[:, :n]).all() if which == "k" else torch.isfinite(lse[:, :n]).all()
        wO, wl, tO, tl = s.reference(2.0 ** -8)
        assert ((O[n:].double() - wO[n:]).abs() <= tO[n:]).all() and torch.isfinite(lse[:, n:]).all()


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q,H", [(4, 2), (4, 4), (5, 6), (40, 2)])
def test_an_e4m3_row_that_is_not_finite_and_later_tokens(which, d, q, H):
    """A row as the append kernel stores it (NaN codes under byte 255): NaN for the new tokens from its own on, the
    same values as before for the earlier ones and for the other head.  8, 16 and 32 rows, and a chunk."""
    for at in (0, q // 2, q - 1):  # which of the request's new tokens
        s = Step([q, 2], [301, 64], H=2 * H, Hkv=2, d=d, ps=32, cache="e4m3", seed=q + H, max_q=q)
        wO, wl, tO, tl = s.reference(*s.rounding())
        j = 301 - q + at
        page, off = s.table_host[0][j // 32], j % 32
        codes, scales = (s.k, s.ks) if which == "k" else (s.v, s.vs)
        codes[page, 1, off], scales[page, 1, off] = 0x7F, 255
        O, lse = s.run()
        sees = torch.zeros(s.T, 2 * H, dtype=torch.bool, device=s.dev)
        sees[at:q, H:] = True
        assert torch.isnan(O[sees]).all()
        assert ((O.double() - wO).abs() <= tO)[~sees].all()
        off_l = ((lse.double() - wl).abs() <= tl).T
        assert off_l[~sees].all() and (torch.isnan(lse.T[sees]).all() if which == "k" else off_l[sees].all())


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_layouts(cache, kind):
    """K and V pages interleaved in one buffer, queries as columns of a wider projection, another softmax scale."""
    q, kv = ([1, 1], [100, 300]) if kind == "decode" else ([40, 130], [100, 300])
    Step(q, kv, H=4, Hkv=2, ps=32, cache=cache, strided=True, q_extra=2 * 2 * 128, scale=0.05, seed=7,
         max_q=1 if kind == "decode" else 0).check()


@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_wide_range_of_scales(kind):
    """E4M3 rows whose exponents span many binades, far above 2^7 too; peaked and flat softmax rows."""
    s = Step([1, 1] if kind == "decode" else [40, 9], [150, 64], cache="e4m3", seed=11,
             max_q=1 if kind == "decode" else 0)
    g = torch.Generator().manual_seed(5)
    s.vs.copy_(torch.randint(100, 160, s.vs.shape, generator=g, dtype=torch.uint8))
    s.ks.copy_(torch.randint(110, 124, s.ks.shape, generator=g, dtype=torch.uint8))
    s.check()


def test_results_do_not_depend_on_the_run():
    """The same call twice gives the same bits (joins happen in a fixed order), whatever the workspace held."""
    for q, kv, mq in (([1] * 5, [9000, 3, 500, 4000, 77], 1), ([64, 1, 30], [5000, 2000, 3000], 0)):
        s = Step(q, kv, H=8, Hkv=2, seed=1, max_q=mq)
        a, la = (x.clone() for x in s.run())
        for i in range(5):
            s.ws.fill_(17 * i)
            b, lb = s.run()
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_captured_step_replays_with_new_lengths():
    """Plan and forward in a CUDA graph; the lengths change between replays."""
    s = Step([1, 1, 1], [100, 200, 300], H=8, Hkv=2, max_q=1, seed=3)
    s.run()
    torch.cuda.synchronize()
    O, lse = torch.zeros_like(s.O), torch.zeros_like(s.lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fl.flamia_paged_plan(s.prob, s.ws)
        fl.flamia_paged_fwd(s.prob, s.q, s.pool, O, lse, s.ws)
    for kv in ([100, 200, 300], [7, 1, 250], [0, 64, 33]):
        s.kv_len = kv
        s.kv.copy_(torch.tensor(kv))
        graph.replay()
        s.run()
        assert torch.equal(O, s.O) and torch.equal(lse, s.lse)
        s.check()


def test_other_streams():
    """Two steps on two streams, each with its own workspace."""
    a, b = Step([1, 1], [3000, 70], H=8, Hkv=2, max_q=1, seed=1), Step([90], [500], H=8, Hkv=2, seed=2)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(sa):
            a.run()
        with torch.cuda.stream(sb):
            b.run()
    torch.cuda.synchronize()
    got = a.O.clone(), b.O.clone()
    a.check()
    b.check()
    assert torch.equal(got[0], a.O) and torch.equal(got[1], b.O)


@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_bad_page_is_reported(kind):
    """A table entry outside the pool sets the status word; other requests are served."""
    s = Step([1, 1] if kind == "decode" else [20, 30], [50, 60], seed=8, max_q=1 if kind == "decode" else 0)
    for bad in (-1, s.n_pages, 2 ** 31 - 1):
        s.table[0, 1] = bad
        O, _ = s.run()
        torch.cuda.synchronize()
        assert fl.flamia_get_device_status(s.ws) == fl.ERR_BAD_PAGE
        s.table[0, 1] = s.table_host[0][1]
        n = s.q_len[0]
        wO, _, tO, _ = s.reference(2.0 ** -8)
        assert ((O[n:].double() - wO[n:]).abs() <= tO[n:]).all()


@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_inconsistent_lengths_write_nothing(kind):
    for field, at, val in (("cu_q", 0, 1), ("cu_q", 1, 10 ** 6), ("cu_q", 2, -5), ("kv", 0, -1), ("kv", 1, 10 ** 8)):
        s = Step([1, 1] if kind == "decode" else [20, 30], [50, 60], max_q=1 if kind == "decode" else 0)
        getattr(s, field)[at] = val
        O, lse = s.run()
        torch.cuda.synchronize()
        assert fl.flamia_get_device_status(s.ws) == fl.ERR_BAD_SEQLENS, (field, at, val)
        assert (O == 77).all() and (lse == 77).all()
    s = Step([3, 1], [50, 60], max_q=2)  # more new tokens than max_q
    O, lse = s.run()
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(s.ws) == fl.ERR_BAD_SEQLENS and (O == 77).all()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["drafts", "chunk", "split"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_later_tokens_reach_no_earlier_row(cache, d, kind, value):
    """A value or key of a new token that is not finite changes nothing in the rows that may not see it."""
    q, kv = {"drafts": ([4, 3], [37, 64]), "chunk": ([200, 60], [400, 60]), "split": ([150, 3], [5000, 64])}[kind]
    kw = dict(H=4, Hkv=2, d=d, ps=16, cache=cache, seed=21, max_q=4 if kind == "drafts" else 0)
    clean = Step(q, kv, **kw)
    cO, cl = clean.run()
    for which, token in (("v", 2), ("v", q[0] - 1), ("k", 1)):
        s = Step(q, kv, **kw)
        j = kv[0] - q[0] + token
        page, off = s.table_host[0][j // 16], j % 16
        if cache == "bf16":
            (s.k if which == "k" else s.v)[page, :, off, 7] = value
        else:
            (s.ks if which == "k" else s.vs)[page, :, off] = 255
        O, lse = s.run()
        other = [i for i in range(s.T) if not token <= i < q[0]]
        # rows that do not see it: as without it (half a step more where an accumulator's last bit moves)
        assert ((O[other].float() - cO[other].float()).abs() <= cO[other].float().abs() * 2.0 ** -7 + 1e-30).all()
        assert torch.equal(lse[:, other], cl[:, other])
        own = O[token:q[0]].float()
        if which == "v":
            assert torch.equal(lse, cl)
            if cache == "bf16":
                assert (own[..., 7] == value).all() if not math.isnan(value) else torch.isnan(own[..., 7]).all()
                rest = [c for c in range(d) if c != 7]
                assert torch.isfinite(own[..., rest]).all()
            else:
                assert torch.isnan(own).all()
        elif cache == "e4m3" or math.isnan(value):
            assert torch.isnan(own).all() and torch.isnan(lse[:, token:q[0]]).all()


@pytest.mark.parametrize("kind", ["decode", "drafts", "chunk"])
def test_infinite_values_stay_infinite(kind):
    """An infinity in V reaches the rows that see it as an infinity, both signs as a NaN, and nothing else."""
    q, kv, mq = {"decode": ([1, 1], [50, 300], 1), "drafts": ([4, 2], [50, 300], 4), "chunk": ([30, 1], [50, 300], 0)}[kind]
    s = Step(q, kv, H=4, Hkv=2, seed=31, max_q=mq)
    page = s.table_host[0][0]
    s.v[page, :, 3, 9], s.v[page, :, 5, 17] = math.inf, -math.inf
    s.v[page, :, 3, 33], s.v[page, :, 6, 33] = math.inf, -math.inf
    s.check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_offsets_past_32_bits(cache, kind):
    """Pages that lie more than 2^32 bytes into the pool, for the append, the decode and the chunk kernel."""
    Hkv, ps, d = 8, 128, 128
    el = 2 if cache == "bf16" else 1
    n_pages = (1 << 32) // (Hkv * ps * d * el) + 40
    kv, mq = ([1, 200, 300], 1) if kind == "decode" else ([90, 200, 300], 90)
    q = [1, 1, 1] if kind == "decode" else [90, 1, 70]
    small = Step(q, kv, H=16, Hkv=Hkv, ps=ps, cache=cache, seed=3, max_q=mq)
    base = n_pages - small.n_pages
    big = [torch.empty(n_pages, Hkv, ps, d, dtype=small.k.dtype, device="cuda") for _ in range(2)]
    for dst, src in zip(big, (small.k, small.v)):
        dst[base:] = src
    scales = []
    if cache == "e4m3":
        for src in (small.ks, small.vs):
            s = torch.full((n_pages, Hkv, ps), 127, dtype=torch.uint8, device="cuda")
            s[base:] = src
            scales.append(s)
    table = torch.where(small.table >= 0, small.table + base, small.table)
    prob = fl.make_paged(small.T, 16, Hkv, d, small.cu_q, small.kv, table, page_size=ps, n_pages=n_pages, max_q=mq,
                         cache_dtype=small.prob.cache_dtype)
    ws = torch.zeros(fl.flamia_paged_workspace_size(prob), dtype=torch.uint8, device="cuda")
    pool = fl.paged_cache(*big, *scales)
    slots = torch.empty(small.T, dtype=torch.int32, device="cuda")
    O, lse = torch.empty_like(small.q).view(small.T, 16, d), torch.empty(16, small.T, device="cuda")
    fl.flamia_paged_plan(prob, ws, slots)
    # the new tokens' rows taken out of their slots and put back by the append
    page, off = slots.long() // ps, slots.long() % ps
    rows = []
    for i, dst in enumerate(big):
        x = dst[page, :, off]
        rows.append(x if cache == "bf16" else torch.ldexp(x.view(torch.float8_e4m3fn).float(), scales[i][page, :, off].int()[..., None] - 127).bfloat16())
        dst[page, :, off] = 0
    fl.flamia_paged_append(prob, rows[0].contiguous(), rows[1].contiguous(), slots, pool, ws)
    fl.flamia_paged_fwd(prob, small.q, pool, O, lse, ws)
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(ws) == fl.OK
    want, wl = small.run()
    assert torch.equal(O, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_workspace_of_another_plan_is_refused(kind):
    """A workspace that was never planned, or planned for another problem: nothing is written, the status says so."""
    s = Step([1, 1] if kind == "decode" else [20, 30], [50, 60], max_q=1 if kind == "decode" else 0)
    O, lse = torch.full((s.T, s.H, s.d), 5.0, dtype=torch.bfloat16, device="cuda"), None
    for prepare in (lambda: s.ws.zero_(), lambda: s.ws.fill_(255).narrow(0, 0, 8).zero_(),
                    lambda: fl.flamia_paged_plan(fl.make_paged(s.T, s.H, s.Hkv, s.d, s.cu_q, s.kv, s.table, page_size=s.ps,
                                                               n_pages=s.n_pages - 1, max_q=s.prob.max_q), s.ws)):
        prepare()
        k = torch.zeros(s.T, s.Hkv, s.d, dtype=torch.bfloat16, device="cuda")
        before = s.k.clone()
        fl.flamia_paged_append(s.prob, k, k, torch.zeros(s.T, dtype=torch.int32, device="cuda"), s.pool, s.ws)
        fl.flamia_paged_fwd(s.prob, s.q, s.pool, O, lse, s.ws)
        torch.cuda.synchronize()
        assert fl.flamia_get_device_status(s.ws) == fl.ERR_INVALID_ARG
        assert (O == 5).all() and torch.equal(before, s.k)
    s.check()


@pytest.mark.parametrize("kind", ["decode", "drafts", "mixed"])
def test_captured_forward_of_each_kernel(kind):
    """Plan and forward captured and replayed, without the log-sum-exp, beside the same calls outside a graph."""
    q, kv, mq = {"decode": ([1, 1], [700, 30], 1), "drafts": ([8, 3], [700, 30], 8),
                 "mixed": ([100, 1, 1, 30], [400, 5000, 0, 30], 0)}[kind]
    s = Step(q, kv, H=8, Hkv=2, cache="e4m3", max_q=mq, seed=12)
    want, _ = s.run()
    O = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fl.flamia_paged_plan(s.prob, s.ws)
        fl.flamia_paged_fwd(s.prob, s.q, s.pool, O, None, s.ws)
        twice = O * 2  # what follows on the stream sees the whole result
    for _ in range(20):
        O.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, want) and torch.equal(twice, want * 2)


def test_what_follows_on_the_stream_waits():
    """The kernel behind a mixed call, whose two kernels overlap, sees all rows of both."""
    s = Step([200, 1, 1, 1, 64], [3000, 9000, 7000, 40, 64], H=8, Hkv=2, ps=64, seed=13)
    want = s.run()[0].clone()
    fl.flamia_paged_plan(s.prob, s.ws)
    for _ in range(30):
        s.O.fill_(0)
        fl.flamia_paged_fwd(s.prob, s.q, s.pool, s.O, None, s.ws)
        assert torch.equal(s.O.clone(), want)


@pytest.mark.parametrize("cache", CACHES)
def test_many_requests(cache):
    """More requests than workers, most of them short; a call without any new token."""
    kv = [1 + (37 * i) % 61 for i in range(700)]
    Step([1] * 700, kv, H=2, Hkv=1, d=64, cache=cache, max_q=1, seed=14).check()
    s = Step([0, 0, 0], [5, 0, 77], cache=cache, pad=4)
    O, lse = s.run()
    assert (O == 77).all() and (lse == 77).all() and fl.flamia_get_device_status(s.ws) == fl.OK
