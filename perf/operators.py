"""The operators that serve a model from a paged key/value cache: what is measured.

Three operators, used one after the other in a serving step:

  pages   block tables and slot maps built on the GPU from request lengths
          (flamia_paged_plan): pages given back and taken from a free stack
  append  new K and V rows into their cache slots (flamia_paged_append): bf16
          pages, or E4M3 codes with one no-clamp power-of-two exponent per
          (token, head) as the quantizer's per-token option writes them
  attend  attention of a chunk of new tokens (one or many per request) over
          the paged cache (flamia_paged_fwd): O and the log-sum-exp of each row

Layouts: q, O [T][H][d] bf16, lse [H][T] fp32, new k and v [T][Hkv][d]; a cache
[n_pages][Hkv][page_size][d] with scale bytes [n_pages][Hkv][page_size];
block tables int32 [n_req][max_pages].  Request r owns the packed rows
[cu_q[r], cu_q[r+1]), the last ones of its kv_len[r] cached tokens; rows behind
the last request are left as they were.
"""
import math
import random

import torch

own = False

DEV = "cuda"
MAX_SCORES = 2 << 30  # scores that the plain form holds at a time


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _attend(name, **kw):
    # n_req requests with q_lo..q_hi new tokens, n_dec more with one, n_idle inactive ones (a captured batch's
    # padding: one row, nothing cached); ctx_lo..ctx_hi tokens cached before; pad rows behind the last request
    c = dict(op="attend", n_req=0, q_lo=1, q_hi=1, n_dec=0, n_idle=0, ctx_lo=0, ctx_hi=0, H=32, Hkv=8, d=128,
             page=64, cache="bf16", causal=True, pad=0, shape=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _append(name, **kw):
    c = dict(op="append", n_req=1, q_lo=1, q_hi=1, n_dec=0, n_idle=0, ctx_lo=0, ctx_hi=0, H=32, Hkv=8, d=128,
             page=64, cache="e4m3", dtype="bf16", pad=0, shape=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _pages(name, **kw):
    # n_done requests that finished (their pages go back), n_cut whose drafted tokens were rejected
    c = dict(op="pages", n_req=1, q_lo=1, q_hi=1, n_dec=0, n_idle=0, n_done=0, n_cut=0, ctx_lo=0, ctx_hi=0, page=16,
             pad=0, shape=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of a served batch: every request grows by a token, a few finish
        _pages("pages decode 64", n_dec=60, n_done=4, ctx_lo=32, ctx_hi=16384, page=16),
        # an admission step of a large server: long prompts enter, hundreds decode, many leave
        _pages("pages admit 1024", n_req=24, q_lo=500, q_hi=8192, n_dec=900, n_done=70, n_cut=30, ctx_lo=0,
               ctx_hi=32768, page=16, pad=77),
        # the K/V rows of one decode step into an 8-bit cache
        _append("append decode 64 e4m3", n_dec=64, ctx_lo=32, ctx_hi=4096, page=64, pad=3),
        # the K/V rows of a 32K-token prefill step (packed prompts) into an 8-bit cache
        _append("append prefill 32k e4m3", n_req=20, q_lo=200, q_hi=4096, ctx_lo=0, ctx_hi=512, page=128),
        # fp32 rows of a small model into a bf16 cache, ragged, with a padded tail
        _append("append ragged f32 bf16", n_req=13, q_lo=1, q_hi=777, ctx_lo=0, ctx_hi=1000, H=16, Hkv=16, d=64,
                page=16, cache="bf16", dtype="f32", pad=29),
        # the smallest call: a handful of short requests, one inactive slot, multi-head
        _attend("decode small", n_dec=5, n_idle=1, ctx_lo=1, ctx_hi=300, H=16, Hkv=16, d=64, page=16),
        # one user with a long document: a single row per head, the work split over the keys
        _attend("decode long 64k", n_dec=1, ctx_lo=65521, ctx_hi=65521, page=64),
        # a served decode batch on the 8-bit cache
        _attend("decode batch 64 e4m3", n_dec=64, ctx_lo=512, ctx_hi=16384, page=16, cache="e4m3"),
        # drafted tokens of speculative decoding checked in one call
        _attend("drafts 16x8 e4m3", n_req=16, q_lo=2, q_hi=8, ctx_lo=1000, ctx_hi=12000, page=32, cache="e4m3"),
        # a chunk of a long prompt over what is cached of it
        _attend("chunk 2k over 32k", n_req=1, q_lo=2048, q_hi=2048, ctx_lo=32768, ctx_hi=32768, page=64),
        # whole prompts, nothing cached before, multi-head, 8-bit cache
        _attend("prefill 4x4k e4m3", n_req=4, q_lo=4096, q_hi=4096, H=16, Hkv=16, page=128, cache="e4m3"),
        # chunked prefill mixed with decoding requests, as a scheduler packs them
        _attend("mixed 3 chunks 48 dec e4m3", n_req=3, q_lo=300, q_hi=1100, n_dec=48, n_idle=1, ctx_lo=64, ctx_hi=16384,
                page=64, cache="e4m3", pad=17),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    most = max((_flops(c) for c in listed()), default=0)
    while True:
        shape = rng.randrange(1, 1 << 30)
        page = rng.choice([16, 32, 64, 128])
        op = rng.choice(["pages", "append", "attend", "attend", "attend"])
        if op == "pages":
            c = _pages(None, n_req=rng.randrange(0, 20), q_lo=1, q_hi=_log(rng, 1, 8192), n_dec=_log(rng, 1, 900),
                       n_done=rng.randrange(0, 60), n_cut=rng.randrange(0, 30), ctx_lo=0, ctx_hi=_log(rng, 16, 32768),
                       page=page, pad=rng.randrange(0, 100), shape=shape)
        else:
            Hkv = rng.choice([1, 2, 4, 8, 16])
            G = rng.choice([1, 2, 3, 4, 5, 8])
            kw = dict(H=Hkv * G, Hkv=Hkv, d=rng.choice([64, 128, 128]), page=page,
                      cache=rng.choice(["bf16", "e4m3"]), pad=rng.choice([0, 0, rng.randrange(1, 64)]), shape=shape)
            if op == "append":
                c = _append(None, n_req=rng.randrange(1, 20), q_lo=1, q_hi=_log(rng, 1, 4096),
                            n_dec=rng.randrange(0, 64), ctx_lo=0, ctx_hi=_log(rng, 1, 2000),
                            dtype=rng.choice(["bf16", "f32"]), **kw)
            else:
                kind = rng.choice(["decode", "drafts", "chunk", "mixed"])
                ctx = _log(rng, 16, 65536)
                kw.update(ctx_lo=max(1, ctx // rng.choice([1, 2, 16])), ctx_hi=ctx)
                if kind == "decode":
                    kw.update(n_dec=_log(rng, 1, 64), n_idle=rng.choice([0, 0, 2]))
                elif kind == "drafts":
                    kw.update(n_req=_log(rng, 1, 32), q_lo=1, q_hi=rng.randrange(2, 9))
                elif kind == "chunk":
                    kw.update(n_req=rng.randrange(1, 5), q_lo=16, q_hi=_log(rng, 16, 4096), ctx_lo=0,
                              causal=rng.random() < 0.8)
                else:
                    kw.update(n_req=rng.randrange(1, 4), q_lo=16, q_hi=_log(rng, 16, 1100), n_dec=_log(rng, 1, 48),
                              n_idle=1)
                c = _attend(None, **kw)
        if _flops(c) <= most and work(c)["bytes"] <= 1.2e9 and sum(_lens(c)[2]) <= 600000:
            return c


def _lens(c):
    """(new tokens, tokens cached before, tokens cached after) of each request."""
    r = random.Random(c["shape"])
    q, old, new = [], [], []

    def ctx():
        lo, hi = c["ctx_lo"], c["ctx_hi"]
        return lo if lo == hi else int(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1 if lo < hi else hi

    for _ in range(c["n_req"]):
        q.append(r.randint(c["q_lo"], c["q_hi"]))
        old.append(ctx())
        new.append(old[-1] + q[-1])
    for _ in range(c["n_dec"]):
        q.append(1)
        old.append(ctx())
        new.append(old[-1] + 1)
    for _ in range(c["n_idle"]):
        q.append(1)
        old.append(0)
        new.append(0)
    for _ in range(c.get("n_done", 0)):
        q.append(0)
        old.append(ctx())
        new.append(0)
    for _ in range(c.get("n_cut", 0)):
        q.append(4)
        old.append(ctx() + 40)
        new.append(old[-1] - r.randint(1, 36) + 4)
    both = list(zip(q, old, new))
    r.shuffle(both)
    return [b[0] for b in both], [b[1] for b in both], [b[2] for b in both]


def _pairs(c):
    """Visible (row, key) pairs of all heads, and the keys that some row sees."""
    q, _, new = _lens(c)
    pairs = keys = 0
    for n, kv in zip(q, new):
        if not c["causal"]:
            pairs += n * kv
            keys += kv if n else 0
        else:
            seen = min(n, kv)  # rows that see a key: the last one sees kv, the one before it kv - 1
            pairs += seen * kv - seen * (seen - 1) // 2
            keys += kv if seen else 0
    return pairs * c["H"], keys


def _flops(c):
    return 4.0 * c["d"] * _pairs(c)[0] if c["op"] == "attend" else 0.0


def work(case):
    c = case
    q, old, new = _lens(c)
    rows = sum(q)
    if c["op"] == "pages":
        ps = c["page"]
        taken = sum(max(0, -(-b // ps) - -(-a // ps)) for a, b in zip(old, new))
        given = sum(max(0, -(-a // ps) - -(-b // ps)) for a, b in zip(old, new))
        # lengths and offsets in, slot map out, each page taken or given back read and written once; a token's own
        # page is read where it was there before
        return {"bytes": 4.0 * (3 * len(q) + 1 + rows + c["pad"] + 2 * taken + 2 * given), "flops": 0.0}
    row = c["Hkv"] * (c["d"] * (2 if c["cache"] == "bf16" else 1) + (0 if c["cache"] == "bf16" else 1))
    if c["op"] == "append":
        return {"bytes": 2.0 * rows * (row + c["Hkv"] * c["d"] * (2 if c["dtype"] == "bf16" else 4)) + 4.0 * rows, "flops": 0.0}
    pairs, keys = _pairs(c)
    return {"bytes": 2.0 * keys * row + rows * c["H"] * (4.0 * c["d"] + 4) + 4.0 * keys / c["page"], "flops": 4.0 * c["d"] * pairs}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
class State:
    pass


def _quantize_rows(x):
    """E4M3 codes (uint8) and UE8M0 bytes of rows [..., d]: the smallest exponent e with max|x| <= 448 2^e."""
    m, e = torch.frexp(x.abs().amax(-1).float())
    e = torch.where(m > 0.875, e - 8, e - 9)  # amax = m 2^e, 448 = 0.875 2^9
    e = torch.where(m == 0, torch.zeros_like(e), e).clamp(-127, 127)
    codes = torch.ldexp(x.float(), -e[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """Rows of E4M3 codes with their UE8M0 bytes, as fp32."""
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), (scales.to(torch.int32) - 127)[..., None])


def _slots(s):
    """Cache slot of each packed row, -1 where it has none."""
    t = torch.arange(s.T, device=DEV)
    r = torch.searchsorted(s.cu_q[1:].contiguous(), t.to(torch.int32), right=True).clamp(max=s.n_req - 1)
    pos = s.kv_len[r] - (s.cu_q[r + 1] - t)
    page = s.block_table[r, (pos // s.page).clamp(0, s.max_pages - 1)]
    live = (t < s.cu_q[-1]) & (pos >= 0)
    return torch.where(live, page * s.page + pos % s.page, torch.full_like(pos, -1)).to(torch.int32)


def prepare(case, seed):
    c, s = case, State()
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + 17)
    q, old, new = _lens(c)
    s.op, s.case, s.page, s.n_req = c["op"], c, c["page"], len(q)
    s.T, s.max_q = sum(q) + c["pad"], max(max(q), 1)
    s.host = (q, old, new)
    ps = s.page
    i32 = dict(dtype=torch.int32, device=DEV)
    s.cu_q = torch.tensor([0] + list(torch.tensor(q).cumsum(0)), **i32)
    s.old_len, s.kv_len = torch.tensor(old, **i32), torch.tensor(new, **i32)
    held = torch.tensor([-(-a // ps) for a in (old if s.op == "pages" else new)])  # pages in the tables now
    need = torch.tensor([-(-max(a, b) // ps) for a, b in zip(old, new)])
    s.max_pages = max(1, int(need.max())) + 3
    n_held = int(held.sum())
    s.n_pages = n_held + max(0, int((need - held).sum())) + 11
    order = torch.randperm(s.n_pages, generator=g, device=DEV).to(torch.int32)
    s.block_table = torch.zeros(s.n_req, s.max_pages, **i32)
    has = torch.arange(s.max_pages)[None, :] < held[:, None]
    s.block_table[has.to(DEV)] = order[:n_held]
    s.free_pages = torch.zeros(s.n_pages, **i32)
    s.free_pages[: s.n_pages - n_held] = order[n_held:]
    s.n_free = torch.tensor([s.n_pages - n_held], **i32)
    if s.op == "pages":
        s.n_free_out = torch.zeros(1, **i32)
        s.slot_map = torch.zeros(s.T, **i32)
    else:
        s.H, s.Hkv, s.d = c["H"], c["Hkv"], c["d"]
        rand = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
        # tokens differ in size, and a few channels stand out, as keys and values of trained models do
        chan = torch.ones(s.Hkv, s.d, device=DEV)
        chan[:, :: 37] = 4.0
        size = lambda *shape: torch.exp(0.3 * rand(*shape))  # noqa: E731
        if s.op == "append":
            dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
            s.k, s.v = ((rand(s.T, s.Hkv, s.d) * size(s.T, s.Hkv, 1) * chan).to(dt) for _ in range(2))
            pools = [torch.zeros(s.n_pages, s.Hkv, ps, s.d, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
        else:
            s.q = (1.5 * rand(s.T, s.H, s.d)).to(torch.bfloat16)
            pools = [rand(s.n_pages, s.Hkv, ps, s.d).mul_(size(s.n_pages, s.Hkv, ps, 1)).mul_(ch[None, :, None, :]).to(torch.bfloat16)
                     for ch in (torch.ones_like(chan), chan)]
            s.O = torch.zeros(s.T, s.H, s.d, device=DEV, dtype=torch.bfloat16)
            s.lse = torch.zeros(s.H, s.T, device=DEV)
            s.slabs = _slabs(c, q, new)
        if c["cache"] == "e4m3":
            (s.k_pool, s.k_scales), (s.v_pool, s.v_scales) = (_quantize_rows(x) for x in pools)
        else:
            (s.k_pool, s.v_pool), s.k_scales, s.v_scales = pools, None, None
        s.slot_map = _slots(s)
        s.live = (s.slot_map >= 0).nonzero()[:, 0]
    if own:
        import precision_causal_attention_token_gb300 as fl
        s.fl = fl
        model = (1, 1, 64) if s.op == "pages" else (s.H, s.Hkv, s.d)
        s.prob = fl.make_paged(s.T, *model, s.cu_q, s.kv_len, s.block_table, page_size=ps, n_pages=s.n_pages,
                               max_q=s.max_q, causal=c.get("causal", True),
                               cache_dtype=fl.E4M3 if c.get("cache") == "e4m3" else fl.BF16,
                               in_dtype=fl.F32 if c.get("dtype") == "f32" else fl.BF16)
        s.ws = torch.zeros(fl.flamia_paged_workspace_size(s.prob), dtype=torch.uint8, device=DEV)
        if s.op != "pages":
            s.kv = fl.paged_cache(s.k_pool, s.v_pool, s.k_scales, s.v_scales)
            fl.flamia_paged_plan(s.prob, s.ws)  # once per step, before the layers
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    s = state
    if own:
        if s.op == "pages":
            s.fl.flamia_paged_plan(s.prob, s.ws, s.slot_map, s.old_len, s.free_pages, s.n_free, s.n_free_out)
        elif s.op == "append":
            s.fl.flamia_paged_append(s.prob, s.k, s.v, s.slot_map, s.kv, s.ws)
        else:
            s.fl.flamia_paged_fwd(s.prob, s.q, s.kv, s.O, s.lse, s.ws)
    elif s.op == "pages":
        _plain_pages(s)
    elif s.op == "append":
        _plain_append(s)
    else:
        for at in s.slabs:
            _plain_attend(s, at)
    if s.op == "pages":
        return {"block_table": s.block_table, "slot_map": s.slot_map, "free_pages": s.free_pages, "n_free": s.n_free_out}
    if s.op == "append":
        if s.k_scales is None:
            return {"k": s.k_pool, "v": s.v_pool}
        return {"k": s.k_pool.view(torch.float8_e4m3fn), "v": s.v_pool.view(torch.float8_e4m3fn), "k_scales": s.k_scales, "v_scales": s.v_scales}
    return {"O": s.O, "lse": s.lse}


def _plain_pages(s):
    """Pages in request order: those that a request gives back go on the free stack, those that it takes come off it."""
    ps = s.page
    before, after = (s.old_len + (ps - 1)) // ps, (s.kv_len + (ps - 1)) // ps
    col = torch.arange(s.max_pages, device=DEV)[None, :]
    given = (col >= after[:, None]) & (col < before[:, None])
    taken = (col >= before[:, None]) & (col < after[:, None])
    stack = torch.cat([s.free_pages, s.free_pages])
    at = s.n_free + given.flatten().cumsum(0) - 1
    stack = stack.scatter(0, torch.where(given.flatten(), at, 2 * s.n_pages - 1), torch.where(given, s.block_table, stack[-1]).flatten())
    top = s.n_free + given.sum()
    kth = (taken.flatten().cumsum(0) - 1).view_as(taken)
    s.block_table.copy_(torch.where(taken, stack[(top - 1 - kth).clamp(min=0)], s.block_table))
    s.n_free_out.copy_(top - taken.sum())
    i = torch.arange(s.n_pages, device=DEV)
    s.free_pages.copy_(torch.where((i >= s.n_free) & (i < s.n_free_out), stack[: s.n_pages], s.free_pages))
    s.slot_map.copy_(_slots(s))


def _plain_append(s):
    slot = s.slot_map[s.live].long()[:, None]
    at = (slot // s.page, torch.arange(s.Hkv, device=DEV)[None, :], slot % s.page)
    for x, pool, scales in ((s.k, s.k_pool, s.k_scales), (s.v, s.v_pool, s.v_scales)):
        if scales is None:
            pool[at] = x[s.live].to(torch.bfloat16)
        else:
            pool[at], scales[at] = _quantize_rows(x[s.live])


def _slabs(c, q, new):
    """Requests whose padded scores are held at a time: like chunks together."""
    slabs, at, most = [], [], MAX_SCORES // c["H"]
    for r in sorted((i for i in range(len(q)) if q[i]), key=lambda i: (q[i], new[i])):
        both = at + [r]
        if at and len(both) * max(q[i] for i in both) * max(new[i] for i in both) > most or len(at) >= 64:
            slabs.append(at)
            both = [r]
        at = both
    found = []
    for b in slabs + [at]:
        mq, mk = max(q[i] for i in b), max(1, max(new[i] for i in b))
        valid = torch.arange(mq)[None, :] < torch.tensor([q[i] for i in b])[:, None]
        found.append((torch.tensor(b, device=DEV), mq, mk, valid.flatten().nonzero()[:, 0].to(DEV)))
    return found


def _plain_attend(s, slab):
    idx, mq, mk, valid = slab  # valid: its rows that are there, of the padded n * mq
    n, G = idx.numel(), s.H // s.Hkv
    start, count, kv = s.cu_q[idx], s.cu_q[idx + 1] - s.cu_q[idx], s.kv_len[idx]
    i, j = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
    rows = (start[:, None] + i).clamp(max=s.T - 1)  # [n, mq]
    page = s.block_table[idx][:, (j // s.page)].long()  # [n, mk]
    there = j < kv[:, None]
    page = torch.where(there, page, 0)

    def cached(pool, scales):
        x = pool[page, :, (j % s.page)[None, :]]  # [n, mk, Hkv, d]
        x = x.float() if scales is None else _values(x, scales[page, :, (j % s.page)[None, :]])
        return torch.where(there[:, :, None, None], x, 0.0).transpose(1, 2)

    qs = s.q[rows].float().view(n, mq, s.Hkv, G, s.d).permute(0, 2, 3, 1, 4).reshape(n, s.Hkv, G * mq, s.d)
    x = (qs @ cached(s.k_pool, s.k_scales).transpose(2, 3)).mul_(1.0 / math.sqrt(s.d)).view(n, s.Hkv, G, mq, mk)
    last = kv[:, None] - count[:, None] + i if s.case["causal"] else kv[:, None] - 1 + 0 * i  # the last key row i sees
    x.masked_fill_((j > last[:, :, None])[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = p.sum(-1)
    o = (p.view(n, s.Hkv, G * mq, mk) @ cached(s.v_pool, s.v_scales)).view(n, s.Hkv, G, mq, s.d)
    o = o / torch.where(l > 0, l, 1.0)[..., None]
    lse = m[..., 0] + l.log()
    at = rows.flatten()[valid].long()
    s.O[at] = o.permute(0, 3, 1, 2, 4).reshape(n * mq, s.H, s.d)[valid].to(torch.bfloat16)
    s.lse[:, at] = lse.permute(0, 3, 1, 2).reshape(n * mq, s.H)[valid].t()


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] == "pages":
        return None  # whole numbers
    if c["op"] == "attend" and _flops(c) > 6e12:
        return None
    global own
    was, own = own, False
    s = prepare(c, seed)
    own = was
    q, _, new = s.host
    table, ps = s.block_table.cpu(), s.page

    def slots(r, n):  # the slots of request r's first n tokens
        t = torch.arange(n)
        return (table[r].long()[t // ps] * ps + t % ps).to(DEV)

    def flat(pool):  # [slot][Hkv][...]
        return pool.transpose(1, 2).reshape(s.n_pages * ps, s.Hkv, *pool.shape[3:])

    if c["op"] == "append":
        out = {}
        for name, x, pool, scales in (("k", s.k, s.k_pool, s.k_scales), ("v", s.v, s.v_pool, s.v_scales)):
            if scales is None:
                val, sc = flat(pool).double(), None
            else:
                val, sc = flat(pool.view(torch.float8_e4m3fn).float()).double(), flat(scales).clone()
            row = 0
            for r, n in enumerate(q):
                have = min(n, new[r])
                if have:
                    at = slots(r, new[r])[new[r] - have:]
                    y = x[row + n - have: row + n].double()
                    if scales is None:
                        val[at] = y
                    else:
                        top = y.abs().amax(-1, keepdim=True)
                        e = torch.where(top > 0, torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448.0)), 0.0)
                        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, torch.where((top > 0) & (top <= 448.0 * torch.exp2(e - 1)), e - 1, e))
                        y = y * torch.exp2(-e)
                        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                        val[at] = torch.round(y / step) * step
                        sc[at] = (e[..., 0] + 127).to(torch.uint8)
                row += n
            shape = (s.n_pages, ps, s.Hkv)
            out[name] = val.view(*shape, s.d).transpose(1, 2).contiguous()
            if scales is not None:
                out[name + "_scales"] = sc.view(shape).transpose(1, 2).contiguous()
        return out

    O, lse = torch.zeros(s.T, s.H, s.d, device=DEV, dtype=torch.float64), torch.zeros(s.H, s.T, device=DEV, dtype=torch.float64)
    G, row = s.H // s.Hkv, 0
    for r, n in enumerate(q):
        kv = new[r]
        if kv == 0:
            lse[:, row:row + n] = -math.inf
            row += n
            continue
        at = slots(r, kv)
        page, off = at // ps, at % ps
        for h in range(s.Hkv if n else 0):
            K, V = s.k_pool[page, h, off], s.v_pool[page, h, off]
            if s.k_scales is None:
                K, V = K.double(), V.double()
            else:
                K, V = (x.view(torch.float8_e4m3fn).double() * torch.exp2(b[page, h, off].double() - 127)[:, None]
                        for x, b in ((K, s.k_scales), (V, s.v_scales)))
            for hq in range(h * G, (h + 1) * G):
                z = (s.q[row:row + n, hq].double() @ K.T) / math.sqrt(s.d)
                if c["causal"]:
                    see = torch.arange(kv, device=DEV)[None, :] <= torch.arange(kv - n, kv, device=DEV)[:, None]
                    z = torch.where(see, z, -math.inf)
                w = torch.logsumexp(z, 1)
                lse[hq, row:row + n] = w
                O[row:row + n, hq] = torch.exp(z - torch.where(w == -math.inf, 0.0, w)[:, None]) @ V
        row += n
    return {"O": O, "lse": lse}
