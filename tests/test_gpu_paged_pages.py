"""Shared pages on the GPU: steps of forks, releases, copies on write and compactions against the model of lists."""
import random

import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged4_ref import packed, quantize4, values4
from paged_pages_ref import Pool, up
from paged_ref import quantize_rows, row_values

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


class Gpu:
    """The model's arrays on the GPU, and the calls."""

    def __init__(self, m, n_req, T, max_q=0, fill=0x5A):
        self.m, self.n, self.T = m, n_req, T
        self.cu, self.kv, self.old = torch.zeros(n_req + 1, **I32), torch.zeros(n_req, **I32), torch.zeros(n_req, **I32)
        self.src, self.slots = torch.zeros(n_req, **I32), torch.zeros(T, **I32)
        self.table, self.refs = torch.tensor(m.table, **I32), torch.tensor(m.refs, **I32)
        self.free = torch.full((m.n_pages,), -5, **I32)
        self.free[:len(m.free)] = torch.tensor(m.free, **I32)
        self.n_free, self.n_copies = torch.tensor([len(m.free)], **I32), torch.zeros(1, **I32)
        self.copies = torch.zeros(max(n_req, m.n_pages), 2, **I32)
        self.prob = fl.make_paged(T, 4, 2, 64, self.cu, self.kv, self.table, page_size=m.ps, n_pages=m.n_pages, max_q=max_q)
        self.ws = torch.full((fl.flamia_paged_workspace_size(self.prob),), fill, dtype=torch.uint8, device="cuda")
        self.pages_ws = torch.full((fl.flamia_paged_pages_workspace_size(self.prob),), fill, dtype=torch.uint8, device="cuda")

    def inputs(self, q, kv, src, old):
        self.cu.copy_(torch.tensor([sum(q[:i]) for i in range(self.n + 1)], dtype=torch.int32))
        for a, b in ((self.kv, kv), (self.src, src), (self.old, old)):
            a.copy_(torch.tensor(b, dtype=torch.int32))

    def step(self, src_given=True):
        fl.flamia_paged_plan_shared(self.prob, self.ws, self.pages_ws, self.slots, self.src if src_given else None, self.old, self.refs,
                                    self.free, self.n_free, self.n_free, self.copies, self.n_copies)
        return fl.flamia_get_device_status(self.ws)

    def compact(self, refs=True):
        fl.flamia_paged_compact(self.prob, self.pages_ws, self.old, self.refs if refs else None, self.free, self.n_free, self.copies,
                                self.n_copies)
        return fl.flamia_get_device_status(self.pages_ws)

    def same(self, copies):
        torch.cuda.synchronize()
        m = self.m
        assert int(self.n_copies) == len(copies) and self.copies[:len(copies)].tolist() == copies
        assert self.refs.tolist() == m.refs
        assert int(self.n_free) == len(m.free) and self.free[:len(m.free)].tolist() == m.free
        assert self.table.tolist() == m.table


def _random_step(r, m, n, T, max_q, beams):
    """Lengths of a step that fits the table's columns."""
    q, kv, src = [], [], []
    cap, left = m.max_pages * m.ps, T
    for i in range(n):
        s = r.randrange(-1, n) if beams and r.random() < 0.7 else i
        old = m.held[s] if s >= 0 else 0
        kind = r.random()
        if kind < 0.1:
            a, b = r.choice([0, 1]), 0  # ends; an idle slot of a captured batch
        else:
            a = 0 if kind < 0.15 else 1 if kind < 0.6 else r.randint(1, max_q)
            kept = max(0, old - r.randint(0, 9)) if r.random() < 0.3 else old  # drafts taken back, a part of a prompt
            b = min(cap, kept + a)
        a = min(a, left)
        left -= a
        q.append(a)
        kv.append(b)
        src.append(s)
    return q, kv, src


@pytest.mark.parametrize("n,pages,cols,ps,max_q,beams", [
    (1, 9, 8, 16, 40, False), (7, 60, 12, 16, 30, True), (5, 40, 30, 32, 200, True), (64, 700, 20, 16, 20, True),
    (300, 2000, 9, 64, 33, True), (17, 20, 40, 16, 17, True), (3, 5000, 2100, 16, 9000, True)])
def test_steps_follow_the_model(n, pages, cols, ps, max_q, beams):
    r = random.Random(n * pages)
    free = list(range(pages))
    r.shuffle(free)
    m = Pool(n, pages, cols, ps, free)
    T = n * max_q + 3
    gpu = Gpu(m, n, T, max_q)
    refused = 0
    for it in range(40 if n < 300 else 12):
        q, kv, src = _random_step(r, m, n, T, max_q, beams)
        gpu.inputs(q, kv, src, m.held)
        before = [x.clone() for x in (gpu.table, gpu.refs, gpu.free, gpu.n_free)]
        copies = m.step(q, kv, src)
        status = gpu.step()
        if copies is None:
            refused += 1
            assert status == fl.ERR_NO_PAGES == fl.flamia_get_device_status(gpu.pages_ws) and (gpu.slots == -1).all() and int(gpu.n_copies) == 0
            assert all(torch.equal(a, b) for a, b in zip((gpu.table, gpu.refs, gpu.free, gpu.n_free), before))
            ends = [0] * n  # room again
            gpu.inputs(ends, [0 if i % 2 else h for i, h in enumerate(m.held)], list(range(n)), m.held)
            copies = m.step(ends, [0 if i % 2 else h for i, h in enumerate(m.held)], list(range(n)))
            status, q, kv = gpu.step(), ends, m.held
        assert status == fl.OK
        gpu.same(copies)
        assert gpu.slots.tolist() == m.slots(q, kv, T)
        if it % 7 == 3:
            gpu.old.copy_(torch.tensor(m.held, dtype=torch.int32))
            moves = m.compact()
            assert gpu.compact() == fl.OK
            gpu.same(moves)
    assert refused or n != 17


def test_as_many_requests_as_there_can_be():
    """8,192 requests, most continued by others or ended, in two steps."""
    n, r = 8192, random.Random(9)
    m = Pool(n, 40000, 4, 16)
    gpu = Gpu(m, n, 4 * n, 4)
    q, kv = [1 + i % 4 for i in range(n)], [20 + i % 29 if i % 5 else 3 for i in range(n)]
    q = [min(a, b) for a, b in zip(q, kv)]
    for src in (list(range(n)), [r.randrange(-1, n) if i % 3 else i for i in range(n)]):
        if m.held != [0] * n:
            kv = [(m.held[s] if s >= 0 else 0) + a for s, a in zip(src, q)]
        gpu.inputs(q, kv, src, m.held)
        seen = m.step(q, kv, src)
        assert gpu.step() == fl.OK
        gpu.same(seen)
        assert gpu.slots.tolist() == m.slots(q, kv, 4 * n)
    gpu.old.copy_(torch.tensor(m.held, dtype=torch.int32))
    moves = m.compact()
    assert gpu.compact() == fl.OK
    gpu.same(moves)


def test_two_streams_at_once():
    """Steps and compactions on two streams with buffers of their own, launched side by side."""
    r = random.Random(4)
    sets = []
    for i in range(2):
        m = Pool(700, 9000, 12, 16)
        sets.append((m, Gpu(m, 700, 700 * 8, 8), torch.cuda.Stream()))
    for it in range(12):
        want = []
        for m, gpu, stream in sets:
            q, kv, src = _random_step(r, m, 700, 700 * 8, 8, True)
            gpu.inputs(q, kv, src, m.held)
            want.append((m.step(q, kv, src), q, kv))
            assert want[-1][0] is not None
        torch.cuda.synchronize()
        for m, gpu, stream in sets:
            with torch.cuda.stream(stream):
                fl.flamia_paged_plan_shared(gpu.prob, gpu.ws, gpu.pages_ws, gpu.slots, gpu.src, gpu.old, gpu.refs, gpu.free, gpu.n_free,
                                            gpu.n_free, gpu.copies, gpu.n_copies)
        torch.cuda.synchronize()
        for (m, gpu, stream), (copies, q, kv) in zip(sets, want):
            assert fl.flamia_get_device_status(gpu.ws) == fl.OK
            gpu.same(copies)
            assert gpu.slots.tolist() == m.slots(q, kv, 700 * 8)


def test_without_sources_each_continues_itself():
    m, T = Pool(2, 9, 4, 16), 30
    gpu = Gpu(m, 2, T)
    for q, kv in (([20, 5], [20, 5]), ([1, 4], [21, 9]), ([0, 1], [0, 10])):
        gpu.inputs(q, kv, [9, 9], m.held)
        copies = m.step(q, kv, [0, 1])
        assert gpu.step(src_given=False) == fl.OK
        gpu.same(copies)


def test_pages_held_beside_the_tables():
    """A count more keeps a page from being freed and from being written to."""
    m = Pool(2, 9, 4, 16)
    gpu = Gpu(m, 2, 30)
    m.step([20, 0], [20, 0], [0, 1])
    gpu.inputs([20, 0], [20, 0], [0, 1], [0, 0])
    gpu.step()
    for page in m.table[0][:2]:
        m.refs[page] += 1
        gpu.refs[page] += 1
    gpu.inputs([1, 0], [21, 0], [0, 1], m.held)
    copies = m.step([1, 0], [21, 0], [0, 1])
    assert len(copies) == 1 and gpu.step() == fl.OK
    gpu.same(copies)
    gpu.inputs([0, 0], [0, 0], [0, 1], m.held)
    copies = m.step([0, 0], [0, 0], [0, 1])
    assert gpu.step() == fl.OK
    gpu.same(copies)
    assert sum(m.refs) == 2 and len(m.free) == 7
    gpu.old.zero_()
    moves = m.compact()
    assert gpu.compact() == fl.OK
    gpu.same(moves)


def _broken(what):
    m = Pool(3, 12, 4, 16)
    gpu = Gpu(m, 3, 64, 40)
    m.step([20, 40, 0], [20, 40, 0], [0, 1, 2])
    gpu.inputs([20, 40, 0], [20, 40, 0], [0, 1, 2], [0, 0, 0])
    assert gpu.step() == fl.OK
    gpu.inputs([1, 0, 1], [21, 0, 41], [0, -1, 1], m.held)
    what(gpu)
    torch.cuda.synchronize()
    return m, gpu


def _set(t, i, v):
    t[i] = v


@pytest.mark.parametrize("name,what,status", [
    ("cu", lambda g: _set(g.cu, 1, 3), fl.ERR_BAD_SEQLENS), ("cu0", lambda g: _set(g.cu, 0, -1), fl.ERR_BAD_SEQLENS),
    ("kv", lambda g: _set(g.kv, 0, 65), fl.ERR_BAD_SEQLENS), ("kv<0", lambda g: _set(g.kv, 2, -1), fl.ERR_BAD_SEQLENS),
    ("old", lambda g: _set(g.old, 1, 65), fl.ERR_BAD_SEQLENS), ("old<0", lambda g: _set(g.old, 1, -2), fl.ERR_BAD_SEQLENS),
    ("src", lambda g: _set(g.src, 2, 3), fl.ERR_BAD_SEQLENS), ("src<-1", lambda g: _set(g.src, 0, -2), fl.ERR_BAD_SEQLENS),
    ("n_free<0", lambda g: _set(g.n_free, 0, -1), fl.ERR_BAD_PAGE), ("n_free", lambda g: _set(g.n_free, 0, 13), fl.ERR_BAD_PAGE),
    ("n_free+", lambda g: _set(g.n_free, 0, 12), fl.ERR_BAD_PAGE), ("no pages", lambda g: (_set(g.n_free, 0, 0), _set(g.kv, 2, 64)), fl.ERR_NO_PAGES),
    ("moved entry", lambda g: _set(g.table[1], 0, 12), fl.ERR_BAD_PAGE), ("moved entry<0", lambda g: _set(g.table[1], 2, -1), fl.ERR_BAD_PAGE),
    ("written entry", lambda g: _set(g.table[0], 1, 1 << 30), fl.ERR_BAD_PAGE), ("counts", lambda g: g.refs.zero_(), fl.ERR_BAD_PAGE)])
def test_bad_steps_move_nothing(name, what, status):
    _, gpu = _broken(what)
    if name == "n_free+":  # a page is freed and the stack is full
        gpu.inputs([0, 0, 0], [0, 0, 0], [0, 1, 2], [20, 40, 0])
    state = (gpu.table, gpu.refs, gpu.free, gpu.n_free)
    before = [x.clone() for x in state]
    assert gpu.step() == status == fl.flamia_get_device_status(gpu.pages_ws)
    assert all(torch.equal(a, b) for a, b in zip(state, before))
    assert (gpu.slots == -1).all() and int(gpu.n_copies) == 0
    # launches on the workspace write nothing
    pool = torch.full((12, 2, 16, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    rows = torch.ones(64, 4, 64, dtype=torch.bfloat16, device="cuda")
    O, lse, cache = torch.full_like(rows, 9.0), torch.full((4, 64), 9.0, device="cuda"), fl.paged_cache(pool, pool)
    fl.flamia_paged_append(gpu.prob, rows[:, :2].contiguous(), rows[:, :2].contiguous(), gpu.slots, cache, gpu.ws)
    fl.flamia_paged_fwd(gpu.prob, rows, cache, O, lse, gpu.ws)
    torch.cuda.synchronize()
    assert (pool == 3).all() and (O == 9).all() and (lse == 9).all()


def test_counts_that_fall_short_end_every_cta_alike():
    """One CTA finds them while others may still be leaving the barrier before: none may wait for those that left."""
    n = 150
    m = Pool(n, 900, 6, 16)
    gpu = Gpu(m, n, 64 * n, 64)
    q = kv = [20 + i % 40 for i in range(n)]
    m.step(q, kv, list(range(n)))
    gpu.inputs(q, kv, list(range(n)), [0] * n)
    assert gpu.step() == fl.OK
    gpu.inputs([1] * n, [k + 1 for k in kv], list(range(n)), m.held)
    table = gpu.table.clone()
    for i in [i for i in range(300) if kv[i % n] % 16]:  # at a page's border a row reads no count
        gpu.refs.copy_(torch.tensor(m.refs, dtype=torch.int32))
        gpu.refs[int(gpu.table[i % n, kv[i % n] // 16])] = 0
        assert gpu.step() == fl.ERR_BAD_PAGE == fl.flamia_get_device_status(gpu.pages_ws)
    assert torch.equal(gpu.table, table) and int(gpu.n_free) == len(m.free) and int(gpu.n_copies) == 0


@pytest.mark.parametrize("what,status", [
    (lambda g: _set(g.old, 0, -1), fl.ERR_BAD_SEQLENS), (lambda g: _set(g.old, 0, 65), fl.ERR_BAD_SEQLENS),
    (lambda g: _set(g.n_free, 0, 13), fl.ERR_BAD_PAGE), (lambda g: _set(g.n_free, 0, -1), fl.ERR_BAD_PAGE),
    (lambda g: _set(g.free, 1, 12), fl.ERR_BAD_PAGE), (lambda g: _set(g.free, 1, -1), fl.ERR_BAD_PAGE),
    (lambda g: _set(g.free, 1, int(g.free[0])), fl.ERR_BAD_PAGE), (lambda g: _set(g.table[0], 1, 12), fl.ERR_BAD_PAGE),
    (lambda g: _set(g.table[1], 0, -3), fl.ERR_BAD_PAGE), (lambda g: _set(g.free, 1, int(g.table[1, 2])), fl.ERR_BAD_PAGE)])
def test_bad_compactions_move_nothing(what, status):
    _, gpu = _broken(lambda g: g.old.copy_(torch.tensor([20, 40, 0], dtype=torch.int32)))
    what(gpu)
    state = (gpu.table, gpu.refs, gpu.free, gpu.n_free)
    before = [x.clone() for x in state]
    assert gpu.compact() == status
    assert all(torch.equal(a, b) for a, b in zip(state, before)) and int(gpu.n_copies) == 0


@pytest.mark.parametrize("n_pages", [1, 31, 32, 33, 16000, 200000])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 0.97, 1.0])
def test_compaction_of_pools_of_any_size(n_pages, share):
    """One request holds all pages in use, in any order; without counts and with them."""
    g = torch.Generator().manual_seed(n_pages)
    ids = torch.randperm(n_pages, generator=g)
    used = int(n_pages * share)
    table = torch.zeros(2, max(1, used) + 2, dtype=torch.int32)
    table[1, :used] = ids[:used].int()
    free = torch.full((n_pages,), 7, dtype=torch.int32)
    free[:n_pages - used] = ids[used:].int()
    refs = torch.zeros(n_pages, dtype=torch.int32)
    refs[ids[:used]] = torch.arange(1, used + 1, dtype=torch.int32)
    leaves, holes = ids[:used][ids[:used] >= used].sort().values, ids[used:][ids[used:] < used].sort().values
    to = torch.arange(n_pages)
    to[leaves] = holes
    want = table.clone()
    want[1, :used] = to[table[1, :used].long()].int()
    for with_refs in (True, False):
        t, f, c, n = table.cuda(), free.cuda(), torch.zeros(n_pages, 2, **I32), torch.tensor([n_pages - used], **I32)
        rf, m, cu, length = refs.cuda(), torch.full((1,), 3, **I32), torch.zeros(3, **I32), torch.tensor([0, used * 16], **I32)
        prob = fl.make_paged(1, 1, 1, 64, cu, length, t, page_size=16, n_pages=n_pages, max_q=1)
        ws = torch.full((fl.flamia_paged_pages_workspace_size(prob),), 0xC3, dtype=torch.uint8, device="cuda")
        fl.flamia_paged_compact(prob, ws, length, rf if with_refs else None, f, n, c, m)
        torch.cuda.synchronize()
        assert fl.flamia_get_device_status(ws) == fl.OK
        assert int(m) == len(leaves) and torch.equal(c[:len(leaves)].cpu(), torch.stack([leaves, holes], 1).int())
        assert torch.equal(t.cpu(), want) and int(n) == n_pages - used
        assert f[:n_pages - used].tolist() == [n_pages - 1 - i for i in range(n_pages - used)] and (f[n_pages - used:] == 7).all()
        moved = torch.zeros_like(refs)
        moved[to[ids[:used]]] = refs[ids[:used]]
        assert torch.equal(rf.cpu(), moved if with_refs else refs)


def _pools(cache, n, Hkv, ps, d, layers, strided, g):
    out = []
    for _ in range(layers):
        byte = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
        width = d * 2 if cache == "bf16" else d if cache == "e4m3" else d // 2
        if strided:
            both = byte(n, 2, Hkv, ps, width)
            k, v = both[:, 0], both[:, 1]
        else:
            k, v = byte(n, Hkv, ps, width), byte(n, Hkv, ps, width)
        if cache == "bf16":
            k, v = k.view(torch.bfloat16), v.view(torch.bfloat16)
        pool = [k, v]
        if cache != "bf16":
            pool += [byte(n, Hkv, ps), byte(n, Hkv, ps)]
        if cache == "e2m1":
            pool += [byte(n, Hkv, ps, d // 16), byte(n, Hkv, ps, d // 16)]
        out.append(pool)
    return out


@pytest.mark.parametrize("cache,dt", [("bf16", fl.BF16), ("e4m3", fl.E4M3), ("e2m1", fl.E2M1)])
@pytest.mark.parametrize("Hkv,ps,d,layers,strided,two", [(1, 16, 64, 1, False, False), (3, 16, 64, 33, False, True), (8, 128, 128, 2, True, False),
                                                         (5, 32, 128, 3, True, True), (2, 64, 64, 70, False, False)])
@pytest.mark.parametrize("count", [0, 1, 9])
def test_copies_are_whole_and_nothing_else_changes(cache, dt, Hkv, ps, d, layers, strided, two, count):
    n, g = 24, torch.Generator(device="cuda").manual_seed(count + layers)
    src = _pools(cache, n, Hkv, ps, d, layers, strided, g)
    dst = _pools(cache, n, Hkv, ps, d, layers, not strided, g) if two else src
    ids = torch.randperm(n, generator=torch.Generator().manual_seed(d))[:2 * count].view(-1, 2)
    copies = torch.full((count + 2, 2), 1 << 30, **I32)  # lines behind the count are not read
    copies[:count] = ids.int()
    words = lambda x: x.contiguous().view(torch.uint8).clone()  # noqa: E731
    want = [[words(x) for x in layer] for layer in dst]
    for s, w in zip(src, want):
        for x, y in zip(s, w):
            y[ids[:, 1].cuda()] = words(x)[ids[:, 0].cuda()]
    cu, kv, table, m = torch.zeros(2, **I32), torch.zeros(1, **I32), torch.zeros(1, 1, **I32), torch.tensor([count], **I32)
    prob = fl.make_paged(1, Hkv, Hkv, d, cu, kv, table, page_size=ps, n_pages=n, cache_dtype=dt)
    ws = torch.zeros(fl.flamia_paged_pages_workspace_size(prob), dtype=torch.uint8, device="cuda")
    a = [fl.paged_cache(*layer) for layer in src]
    b = [fl.paged_cache(*layer) for layer in dst] if two else a
    fl.flamia_paged_copy(prob, a, b, copies, m, ws)
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(ws) == fl.OK
    for layer, w in zip(dst, want):
        for x, y in zip(layer, w):
            assert torch.equal(words(x), y)


def test_copies_out_of_range_are_skipped():
    k = torch.arange(6, device="cuda").to(torch.bfloat16)[:, None, None, None].expand(6, 1, 16, 64).contiguous()
    v, cu, kv, table = -k, torch.zeros(2, **I32), torch.zeros(1, **I32), torch.zeros(1, 1, **I32)
    prob = fl.make_paged(1, 1, 1, 64, cu, kv, table, page_size=16, n_pages=6)
    ws = torch.zeros(fl.flamia_paged_pages_workspace_size(prob), dtype=torch.uint8, device="cuda")
    c = [fl.paged_cache(k, v)]
    pairs = torch.tensor([[0, 6], [-1, 1], [2, 3], [6, 4], [4, -2]], **I32)
    fl.flamia_paged_copy(prob, c, c, pairs, torch.tensor([5], **I32), ws)
    assert fl.flamia_get_device_status(ws) == fl.ERR_BAD_PAGE
    assert k[:, 0, 0, 0].tolist() == [0, 1, 2, 2, 4, 5] and v[:, 0, 15, 63].tolist() == [0, -1, -2, -2, -4, -5]
    for count in (6, -1):
        fl.flamia_clear_device_status(ws)
        n = torch.tensor([count], **I32)
        fl.flamia_paged_copy(prob, c, c, pairs[:5], n, ws)
        assert fl.flamia_get_device_status(ws) == fl.ERR_INVALID_ARG
    assert k[:, 0, 0, 0].tolist() == [0, 1, 2, 2, 4, 5]


class Server:
    """PagedCall with shared pages and, on the host, each request's rows."""

    def __init__(self, cache, n_req, T, *, H=4, Hkv=2, d=64, ps=16, n_pages=64, max_pages=12, layers=2, max_q=0):
        self.dt = {"bf16": fl.BF16, "e4m3": fl.E4M3, "e2m1": fl.E2M1}[cache]
        self.pc = fl.PagedCall(n_req, T, H, Hkv, d, ps, n_pages, max_pages, layers=layers, max_q=max_q, cache_dtype=self.dt, shared=True)
        self.cache, self.n, self.T, self.H, self.Hkv, self.d, self.layers = cache, n_req, T, H, Hkv, d, layers
        self.rows = [[(torch.zeros(0, Hkv, d), torch.zeros(0, Hkv, d))] * n_req for _ in range(layers)]
        self.g = torch.Generator().manual_seed(n_req)

    def stored(self, x):
        if self.cache == "bf16":
            return x.double()
        if self.cache == "e4m3":
            return row_values(*quantize_rows(x))
        c, b, s = quantize4(x)
        return values4(packed(c), b, s)

    def step(self, q, kv, src, cu=None, lens=None, call=None):
        pc, dev = self.pc, "cuda"
        cu_h = [sum(q[:i]) for i in range(self.n + 1)]
        data = [tuple(torch.randn(self.T, h, self.d, generator=self.g).bfloat16() for h in (self.Hkv, self.Hkv, self.H)) for _ in range(self.layers)]
        pc.plan(torch.tensor(cu_h, **I32), torch.tensor(kv, **I32), None if src is None else torch.tensor(src, **I32))
        src = list(range(self.n)) if src is None else src
        for layer in range(self.layers):
            k, v, x = data[layer]
            pc.append(layer, k.to(dev), v.to(dev))
            O, lse = pc.attend(layer, x.to(dev))
            torch.cuda.synchronize()
            assert fl.flamia_get_device_status(pc.ws) == fl.OK and fl.flamia_get_device_status(pc.pages_ws) == fl.OK
            before, now = self.rows[layer], []
            for r in range(self.n):
                kept = max(0, kv[r] - q[r])
                old = before[src[r]] if src[r] >= 0 else (torch.zeros(0, self.Hkv, self.d),) * 2
                at = slice(cu_h[r] + (q[r] - min(q[r], kv[r])), cu_h[r + 1])
                now.append(tuple(torch.cat([a[:kept].double(), self.stored(b[at])]) for a, b in zip(old, (k, v))))
                K, V = now[-1]
                assert K.shape[0] == kv[r]
                if not q[r] or not kv[r]:
                    continue
                see = torch.arange(kv[r])[None] <= torch.arange(kv[r] - q[r], kv[r])[:, None]
                for h in range(self.H):
                    hk = h * self.Hkv // self.H
                    z = torch.where(see, x[cu_h[r]:cu_h[r + 1], h].double() @ K[:, hk].T / self.d ** 0.5, -torch.inf)
                    w = torch.softmax(z, 1)
                    # bf16 weights (2^-8) and result (2^-8), and 2^-13 for scores in fp32
                    tol = 2.0 ** -8 * (w @ V[:, hk]).abs() + (2.0 ** -8 + 2.0 ** -13) * 2 * (w @ V[:, hk].abs())
                    got = O[cu_h[r]:cu_h[r + 1], h].double().cpu()
                    assert ((got - w @ V[:, hk]).abs() <= tol).all(), (r, h)
            self.rows[layer] = now


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
def test_serving_with_shared_pages(cache):
    """A cached prompt, answers sampled from it, beams that reorder, drafts taken back, requests that end, a compaction."""
    s = Server(cache, 6, 64)
    s.step([37, 20, 0, 0, 0, 0], [37, 20, 0, 0, 0, 0], None)
    s.step([0, 1, 3, 1, 0, 0], [37, 21, 40, 38, 0, 0], [0, 1, 0, 0, -1, -1])   # two start from the cached prompt
    s.step([0, 1, 1, 1, 1, 1], [37, 22, 41, 39, 41, 41], [0, 1, 2, 3, 2, 2])   # one goes on as three beams
    for perm in ([0, 1, 4, 3, 2, 2], [0, 1, 2, 3, 2, 4], [0, 5, 5, 3, 5, 1]):
        kv = [37] + [s.rows[0][p][0].shape[0] + 1 for p in perm[1:]]
        s.step([0, 1, 1, 1, 1, 1], kv, perm)
    s.pc.compact()
    used = 64 - int(s.pc.n_free)
    assert all(int(s.pc.block_table[r, k]) < used for r in range(6) for k in range(up(int(s.pc.held_len[r]), 16)))
    n = [r[0].shape[0] for r in s.rows[0]]
    s.step([8, 4, 0, 1, 8, 0], [n[0] + 8, n[1] + 1, 0, n[3] + 1, n[4] + 8, 0], None)  # drafts; two end
    n = [r[0].shape[0] for r in s.rows[0]]
    s.step([2, 1, 30, 1, 2, 1], [n[0] - 5, n[1] + 1, 30 + 20, n[3] + 1, n[4] - 6, n[3] + 1], [0, 1, 0, 3, 4, 3])
    s.pc.compact()
    n = [r[0].shape[0] for r in s.rows[0]]
    s.step([1] * 6, [x + 1 for x in n], None)
    s.step([0] * 6, [0] * 6, [-1] * 6)
    assert int(s.pc.n_free) == 64 and int(s.pc.refs.abs().sum()) == 0


def test_captured_beam_steps():
    """One captured step, replayed with other lengths and parents, against eager steps on a second set of buffers."""
    n, T = 4, 8
    made = [fl.PagedCall(n, T, 4, 2, 64, 16, 80, 12, shared=True, max_q=2) for _ in range(2)]
    cu, kv, src = torch.arange(n + 1, **I32), torch.zeros(n, **I32), torch.zeros(n, **I32)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v, q = (torch.zeros(T, h, 64, dtype=torch.bfloat16, device="cuda") for h in (2, 2, 4))

    def step(pc):
        pc.plan(cu, kv, src)
        pc.append(0, k, v)
        return pc.attend(0, q)

    side = torch.cuda.Stream()
    kv.fill_(1)
    src.copy_(torch.arange(n, **I32))
    for pc in made:
        step(pc)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = step(made[0])
    r = random.Random(5)
    for it in range(2, 60):
        kv.fill_(it)
        src.copy_(torch.tensor([r.randrange(n) for _ in range(n)], dtype=torch.int32))
        for x in (k, v, q):
            x.normal_(generator=g)
        graph.replay()
        want = step(made[1])
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a[:n] if a.dim() == 3 else a[:, :n], b[:n] if b.dim() == 3 else b[:, :n])
        for name in ("block_table", "refs", "n_free", "copies", "n_copies", "held_len", "k", "v"):
            assert torch.equal(getattr(made[0], name), getattr(made[1], name)), name
        assert fl.flamia_get_device_status(made[0].ws) == fl.OK
