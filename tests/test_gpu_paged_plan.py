"""flamia_paged_plan (block tables, free stack, slot map) and
flamia_paged_append against list models."""
import math
import random

import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged_ref import model_plan, pages_of, quantize_rows

pytestmark = pytest.mark.gpu


def _step(old, new, q, ps, *, seed=0, T=None, extra=5, H=2, Hkv=2, d=64, max_q=0, manage=True):
    rng = random.Random(seed)
    n = len(q)
    T = sum(q) if T is None else T
    max_pages = max(pages_of(max(a, b), ps) for a, b in zip(old, new)) + 2
    held = sum(pages_of(a, ps) for a in old)
    n_pages = held + sum(max(0, pages_of(b, ps) - pages_of(a, ps)) for a, b in zip(old, new)) + extra
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table = [[-9] * max_pages for _ in range(n)]
    for r in range(n):
        for i in range(pages_of(old[r], ps)):
            table[r][i] = ids.pop()
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(table=torch.tensor(table, **i32), cu=torch.tensor([sum(q[:i]) for i in range(n + 1)], **i32),
             new=torch.tensor(new, **i32), old=torch.tensor(old, **i32),
             free=torch.tensor(ids + [-3] * (n_pages - len(ids)), **i32), n_free=torch.tensor([len(ids)], **i32),
             out=torch.full((1,), -1, **i32), slots=torch.full((max(1, T),), -7, **i32))
    s["prob"] = fl.make_paged(max(1, T), H, Hkv, d, s["cu"], s["new"], s["table"], page_size=ps, n_pages=n_pages,
                              max_q=max_q)
    s["ws"] = torch.full((fl.flamia_paged_workspace_size(s["prob"]),), 0x5A, dtype=torch.uint8, device="cuda")
    s["want"] = model_plan(table, ids, old, new, q, ps, max(1, T)) if extra >= 0 else None
    s["ids"] = ids
    return s


def _run(s):
    fl.flamia_paged_plan(s["prob"], s["ws"], s["slots"], s["old"], s["free"], s["n_free"], s["out"])
    torch.cuda.synchronize()
    return fl.flamia_get_device_status(s["ws"])


def _check(s):
    table, free, slots = s["want"]
    assert s["table"].tolist() == table
    n = int(s["out"])
    assert n == len(free)
    # below the old top the stack keeps its words; what is left of it is the model's stack
    assert s["free"][:n].tolist() == free
    assert s["slots"].tolist() == slots


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("seed", range(6))
def test_grow_and_shrink(ps, seed):
    rng = random.Random(seed * 100 + ps)
    n = [1, 3, 40, 200, 700, 1500][seed]
    old = [rng.choice([0, 0, rng.randrange(1, 40), rng.randrange(1, 1000)]) for _ in range(n)]
    q = [rng.choice([0, 1, 1, rng.randrange(1, 200)]) for _ in range(n)]
    new = [rng.choice([a + b, a + b, max(0, a - rng.randrange(0, 90)) + b, 0]) for a, b in zip(old, q)]
    s = _step(old, new, q, ps, seed=seed, T=sum(q) + 13)
    for _ in range(2):  # n_free is an input: the call can be repeated
        assert _run(s) == fl.OK
        _check(s)


def test_one_token_steps_and_reuse():
    """All requests end and their pages serve the next ones."""
    s = _step([100, 30, 64], [0, 0, 0], [0, 0, 0], 16, T=1)
    assert _run(s) == fl.OK
    _check(s)
    s = _step([100, 30, 0, 0], [0, 0, 90, 50], [0, 0, 90, 50], 16, extra=0)
    assert _run(s) == fl.OK
    _check(s)


def test_free_count_in_place():
    s = _step([5, 100, 40], [50, 0, 41], [45, 0, 1], 16)
    fl.flamia_paged_plan(s["prob"], s["ws"], s["slots"], s["old"], s["free"], s["n_free"], s["n_free"])
    s["out"] = s["n_free"]
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(s["ws"]) == fl.OK
    _check(s)


def test_table_given_by_the_caller():
    s = _step([40, 3, 17], [40, 3, 17], [40, 1, 2], 16, T=50)
    before = s["table"].clone()
    fl.flamia_paged_plan(s["prob"], s["ws"], s["slots"])
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(s["ws"]) == fl.OK
    assert torch.equal(before, s["table"]) and s["slots"].tolist() == s["want"][2]


def test_most_requests():
    n = 8192
    rng = random.Random(1)
    old = [rng.randrange(0, 60) for _ in range(n)]
    q = [rng.randrange(0, 3) for _ in range(n)]
    s = _step(old, [a + b for a, b in zip(old, q)], q, 16, T=sum(q) + 1)
    assert _run(s) == fl.OK
    _check(s)


def test_too_few_pages_changes_nothing():
    s = _step([16, 10], [160, 170], [144, 160], 16, extra=-1)
    before = s["table"].clone(), s["free"].clone()
    assert _run(s) == fl.ERR_NO_PAGES
    assert torch.equal(before[0], s["table"]) and torch.equal(before[1], s["free"])
    assert int(s["out"]) == int(s["n_free"]) and (s["slots"] == -1).all()
    # launches that use the workspace write nothing
    pool = torch.full((s["prob"].n_pages, 2, 16, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(s["prob"].T, 2, 64, dtype=torch.bfloat16, device="cuda")
    O = torch.full_like(k, 9.0)
    s["slots"].fill_(0)
    kv = fl.paged_cache(pool, pool.clone())
    fl.flamia_paged_append(s["prob"], k, k, s["slots"], kv, s["ws"])
    fl.flamia_paged_fwd(s["prob"], k, kv, O, None, s["ws"])
    torch.cuda.synchronize()
    assert (pool == 5).all() and (O == 9).all()


@pytest.mark.parametrize("what", ["n_free negative", "n_free large", "old negative", "old long", "no room"])
def test_inconsistent_state_changes_nothing(what):
    s = _step([160, 40], [16, 41], [1, 1], 16)
    if what.startswith("n_free"):
        s["n_free"].fill_(-1 if "neg" in what else s["prob"].n_pages + 1)
        want = fl.ERR_BAD_PAGE
    elif what == "no room":  # nine pages come back to a stack that has room for five
        s["n_free"].fill_(s["prob"].n_pages - 5)
        want = fl.ERR_BAD_PAGE
    else:
        s["old"][0] = -1 if "neg" in what else 10 ** 7
        want = fl.ERR_BAD_SEQLENS
    before = s["table"].clone(), s["free"].clone(), int(s["n_free"])
    assert _run(s) == want
    assert torch.equal(before[0], s["table"]) and torch.equal(before[1], s["free"]) and int(s["out"]) == before[2]
    assert (s["slots"] == -1).all()


def test_bad_page_ids_become_no_slot():
    s = _step([40, 3], [40, 20], [4, 17], 16)
    s["table"][0, 2] = s["prob"].n_pages  # request 0's tokens 36..39 lie in page 2
    s["free"][:int(s["n_free"])] = -4      # what request 1 takes
    assert _run(s) == fl.OK
    slots = s["slots"].tolist()
    assert slots[:4] == [-2] * 4
    assert slots[4:17] == s["want"][2][4:17] and slots[17:] == [-2] * 4
    pool = torch.full((s["prob"].n_pages, 2, 16, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(s["prob"].T, 2, 64, dtype=torch.bfloat16, device="cuda")
    fl.flamia_paged_append(s["prob"], k, k, s["slots"], fl.paged_cache(pool, pool.clone()), s["ws"])
    torch.cuda.synchronize()
    assert fl.flamia_get_device_status(s["ws"]) == fl.ERR_BAD_PAGE
    assert int((pool == 0).all(-1).all(1).sum()) == 13


# ------------------------------------------------------------------ append
def _append(cache, dtype, d, Hkv, ps, n_slots, T, *, extra=0, seed=0, live=None, strided=False):
    g = torch.Generator().manual_seed(seed)
    live = T if live is None else live
    n_pages = -(-n_slots // ps)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(cu=torch.tensor([0, live], **i32), kv=torch.tensor([live], **i32))
    s["table"] = torch.arange(max(1, pages_of(live, ps)), **i32)[None].contiguous() % n_pages
    row = Hkv * d + extra
    s["x"] = [(torch.randn(T, row, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g))).to(dtype).cuda()
              for _ in range(2)]
    slots = torch.randperm(n_pages * ps, generator=g)[:T].int()
    s["slots"] = slots.cuda()
    fill = torch.uint8 if cache == "e4m3" else torch.bfloat16
    s["pools"] = [torch.full((n_pages, Hkv, ps, d), 3, dtype=fill, device="cuda") for _ in range(2)]
    if strided:
        both = torch.full((n_pages, 2, Hkv, ps, d), 3, dtype=fill, device="cuda")
        s["pools"] = [both[:, 0], both[:, 1]]
    s["scales"] = [torch.full((n_pages, Hkv, ps), 9, dtype=torch.uint8, device="cuda") for _ in range(2)] if cache == "e4m3" else [None, None]
    s["prob"] = fl.make_paged(T, Hkv, Hkv, d, s["cu"], s["kv"], s["table"], page_size=ps, n_pages=n_pages,
                              cache_dtype=fl.E4M3 if cache == "e4m3" else fl.BF16,
                              in_dtype=fl.BF16 if dtype == torch.bfloat16 else fl.F32, kv_stride=row if extra else 0)
    s["ws"] = torch.empty(fl.flamia_paged_workspace_size(s["prob"]), dtype=torch.uint8, device="cuda")
    s["live"], s["d"], s["Hkv"], s["ps"] = live, d, Hkv, ps
    return s


def _run_append(s):
    fl.flamia_paged_plan(s["prob"], s["ws"])
    fl.flamia_paged_append(s["prob"], s["x"][0], s["x"][1], s["slots"],
                           fl.paged_cache(*s["pools"], *s["scales"]), s["ws"])
    torch.cuda.synchronize()


def _want_append(s):
    out = []
    for x, pool, scales in zip(s["x"], s["pools"], s["scales"]):
        w = torch.full(pool.shape, 3, dtype=pool.dtype)
        ws = None if scales is None else torch.full(scales.shape, 9, dtype=torch.uint8)
        x = x.cpu()[:, :s["Hkv"] * s["d"]].view(-1, s["Hkv"], s["d"])
        codes, sc = (x.to(torch.bfloat16), None) if scales is None else quantize_rows(x)
        for t, slot in enumerate(s["slots"].tolist()[:s["live"]]):
            if 0 <= slot < pool.shape[0] * s["ps"]:
                w[slot // s["ps"], :, slot % s["ps"]] = codes[t]
                if sc is not None:
                    ws[slot // s["ps"], :, slot % s["ps"]] = sc[t]
        out.append((w, ws))
    return out


def _check_append(s):
    for (w, ws), pool, scales in zip(_want_append(s), s["pools"], s["scales"]):
        assert torch.equal(pool.cpu(), w)
        assert scales is None or torch.equal(scales.cpu(), ws)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,Hkv,ps", [(64, 1, 16), (128, 3, 32), (64, 8, 128), (128, 8, 64)])
@pytest.mark.parametrize("T", [1, 37, 1000])
def test_append(cache, dtype, d, Hkv, ps, T):
    s = _append(cache, dtype, d, Hkv, ps, 2 * T + 20, T, seed=T)
    _run_append(s)
    _check_append(s)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_append_strided_padded_and_skipped(cache):
    """Rows of a wider projection, interleaved pages, rows without a slot, rows behind the last request."""
    s = _append(cache, torch.bfloat16, 128, 4, 16, 300, 100, extra=64, live=90, strided=True)
    s["slots"][::7] = -1
    _run_append(s)
    assert fl.flamia_get_device_status(s["ws"]) == fl.OK
    _check_append(s)


def test_append_slot_outside_the_pool():
    s = _append("e4m3", torch.float32, 64, 2, 16, 64, 20)
    s["slots"][3], s["slots"][4], s["slots"][5] = 64, 2 ** 31 - 1, -2 ** 31
    _run_append(s)
    assert fl.flamia_get_device_status(s["ws"]) == fl.ERR_BAD_PAGE
    _check_append(s)


def test_append_corner_values():
    """Zero rows, exact powers, the largest and smallest magnitudes; rows with a NaN or an infinity read as NaN."""
    s = _append("e4m3", torch.float32, 64, 1, 16, 64, 16)
    x = s["x"][0].view(16, 64)
    x[0] = 0
    x[1] = -0.0
    x[2] = 448.0
    x[3] = 448.0000305
    x[4] = torch.finfo(torch.float32).max
    x[5] = 1e-45
    x[6] = 2.0 ** -130
    x[7, 1:] = 2.0 ** -120
    x[8, 3] = math.nan
    x[9, 3] = math.inf
    x[10, 3] = -math.inf
    x[11] = 2.0 ** -126
    s["x"][1].copy_(s["x"][0])
    _run_append(s)
    keep = [i for i in range(16) if i not in (8, 9, 10)]
    for pool, scales in zip(s["pools"], s["scales"]):
        codes, sc = quantize_rows(x.cpu()[keep].view(-1, 1, 64))
        for i, t in enumerate(keep):
            slot = int(s["slots"][t])
            assert torch.equal(pool[slot // 16, 0, slot % 16].cpu(), codes[i, 0]), t
            assert int(scales[slot // 16, 0, slot % 16]) == int(sc[i, 0]), t
        for t in (8, 9, 10):
            slot = int(s["slots"][t])
            assert int(scales[slot // 16, 0, slot % 16]) == 255


def test_append_writes_the_exact_options_bytes():
    """Codes and scale bytes are those of flamia_quantize with `exact` for the same K and V."""
    T, H, d = 70, 2, 128
    s = _append("e4m3", torch.bfloat16, d, H, 16, 128, T, seed=3)
    _run_append(s)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    tc = fl.TrainCall(T, H, H, d, cu, exact=True)
    k, v = (x.view(T, H, d) for x in s["x"])
    tc.plan()
    fl.flamia_quantize(tc.prob, fl.ROLE_QKV, [k, k, v], None, [tc.opq, tc.opk, tc.opv], None, tc.ws)
    slot = s["slots"].long()
    for pool, scales, codes, sc in zip(s["pools"], s["scales"], (tc.k_codes, tc.v_codes), (tc.k_scales, tc.v_scales)):
        assert torch.equal(pool[slot // 16, :, slot % 16], codes)
        assert torch.equal(scales[slot // 16, :, slot % 16], sc.t())
