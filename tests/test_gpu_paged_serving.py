"""A run of the paged-cache operators together, as a server uses them: prompts
come in in chunks beside decoding requests, drafted tokens are taken back,
requests end and their pages serve others.  Each step's attention against plain
attention in 64 bits over the rows that were put in."""
import math
import random

import pytest
import torch

import precision_causal_attention_token_gb300 as fl
from paged_ref import HALF_BF16, quantize_rows, row_values

pytestmark = pytest.mark.gpu


class Server:
    """PagedCall and, on the host, what each request's tokens are."""

    def __init__(self, n_req, T, cache, *, H=8, Hkv=2, d=64, ps=16, n_pages=60, max_pages=20, layers=2, max_q=0, seed=0):
        self.call = fl.PagedCall(n_req, T, H, Hkv, d, ps, n_pages, max_pages, layers=layers, max_q=max_q,
                                 cache_dtype=fl.BF16 if cache == "bf16" else fl.E4M3)
        self.cache, self.n_req, self.T, self.H, self.Hkv, self.d, self.layers = cache, n_req, T, H, Hkv, d, layers
        self.rows = [[([], []) for _ in range(n_req)] for _ in range(layers)]  # k, v rows of each request
        self.g = torch.Generator().manual_seed(seed)

    def inputs(self):
        r = lambda h: torch.randn(self.T, h, self.d, generator=self.g).bfloat16()  # noqa: E731
        return [(1.5 * r(self.H), r(self.Hkv), r(self.Hkv)) for _ in range(self.layers)]

    def remember(self, q_len, kv_len, inputs):
        for layer, (_, k, v) in enumerate(inputs):
            row = 0
            for r, n in enumerate(q_len):
                ks, vs = self.rows[layer][r]
                keep = max(0, kv_len[r] - n)
                del ks[keep:], vs[keep:]
                have = min(n, kv_len[r])
                for i in range(n - have, n):
                    ks.append(k[row + i])
                    vs.append(v[row + i])
                row += n

    def check(self, layer, q, q_len, kv_len, O, lse):
        G, row = self.H // self.Hkv, 0
        for r, n in enumerate(q_len):
            ks, vs = self.rows[layer][r]
            assert len(ks) == kv_len[r]
            for i in range(n):
                pos = kv_len[r] - n + i
                t = row + i
                if pos < 0:
                    assert (O[t] == 0).all() and (lse[:, t] == -math.inf).all()
                    continue
                K, V = torch.stack(ks[:pos + 1]).double(), torch.stack(vs[:pos + 1]).double()  # [n, Hkv, d]
                if self.cache == "e4m3":
                    K, V = row_values(*quantize_rows(K)), row_values(*quantize_rows(V))
                for h in range(self.H):
                    x = K[:, h // G] @ q[t, h].double() / math.sqrt(self.d)
                    size = float((K[:, h // G].abs() @ q[t, h].double().abs()).max()) / math.sqrt(self.d)
                    w = torch.softmax(x, 0)
                    want, A = w @ V[:, h // G], w @ V[:, h // G].abs()
                    err = 2 * (size * (self.d + 4) * 2.0 ** -23 + 2.0 ** -21)
                    # output rounding, weights rounded to bf16 once at most, scores (as in paged_ref)
                    tol = HALF_BF16 * want.abs() + 1.02 * A * (err + HALF_BF16) + 2.0 ** -30
                    assert ((O[t, h].double() - want).abs() <= tol).all(), (r, i, h)
                    assert abs(float(lse[h, t]) - float(torch.logsumexp(x, 0))) <= err + 2.0 ** -18, (r, i, h)
            row += n

    def step(self, q_len, kv_len, run=None):
        cu = torch.tensor([sum(q_len[:i]) for i in range(self.n_req + 1)], dtype=torch.int32)
        kv = torch.tensor(kv_len, dtype=torch.int32)
        ins = self.inputs()
        got = (run or self.run)(cu, kv, ins)
        torch.cuda.synchronize()
        assert int(self.call.status) == fl.OK, fl.status_string(int(self.call.status))
        self.remember(q_len, kv_len, ins)
        for layer, (O, lse) in enumerate(got):
            self.check(layer, ins[layer][0], q_len, kv_len, O.cpu(), lse.cpu())

    def run(self, cu, kv, ins):
        c, got = self.call, []
        c.plan(cu.cuda(), kv.cuda())
        for layer, (q, k, v) in enumerate(ins):
            c.append(layer, k.cuda(), v.cuda())
            O, lse = c.attend(layer, q.cuda())
            got.append((O.clone(), lse.clone()))
        return got

    def pages_are_whole(self, kv_len):
        """No page is lost, shared or doubled."""
        c, ps = self.call, self.call.page_size
        n_free, table = int(c.n_free), c.block_table.tolist()
        held = [p for r in range(self.n_req) for p in table[r][:-(-kv_len[r] // ps)]]
        assert sorted(c.free_pages[:n_free].tolist() + held) == list(range(c.n_pages))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_prompts_decoding_drafts_and_reuse(cache):
    s = Server(4, 80, cache, seed=1)
    steps = [([40, 0, 3, 0], [40, 0, 3, 0]),       # two prompts, one in its first chunk
             ([30, 1, 1, 0], [70, 1, 4, 0]),       # its second chunk beside decoding
             ([1, 1, 4, 50], [71, 2, 8, 50]),      # drafted tokens
             ([1, 1, 2, 1], [72, 3, 7, 51]),       # three of them taken back, two new
             ([0, 1, 1, 1], [0, 4, 8, 52]),        # request 0 ends
             ([60, 1, 1, 0], [60, 5, 9, 0]),       # its pages and request 3's serve the next prompt
             ([1, 1, 1, 1], [61, 6, 10, 0])]       # an inactive slot with a row of its own
    for q_len, kv_len in steps:
        s.step(q_len, kv_len)
        s.pages_are_whole(kv_len)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_captured_decode_steps(cache):
    """A decode step in a CUDA graph, replayed as the requests grow, end and start."""
    s = Server(3, 3, cache, max_q=1, n_pages=20, max_pages=8, seed=2)
    static = [tuple(x.cuda() for x in layer) for layer in s.inputs()]
    cu, kv = torch.arange(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    out = []

    def body():
        out.clear()
        c = s.call
        c.plan(cu, kv)
        for layer, (q, k, v) in enumerate(static):
            c.append(layer, k, v)
            O, lse = c.attend(layer, q)
            out.append((O.clone(), lse.clone()))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        body()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()

    def replay(cu_h, kv_h, ins):
        kv.copy_(kv_h)
        for dst, src in zip(static, ins):
            for a, b in zip(dst, src):
                a.copy_(b)
        graph.replay()
        return out

    lens = [0, 0, 0]
    for i in range(40):
        lens = [0 if i in (17, 30) and r == 1 else n + 1 for r, n in enumerate(lens)]
        s.step([1, 1, 1], lens, replay)
        s.pages_are_whole(lens)


def test_pool_runs_out_and_recovers():
    s = Server(2, 200, "bf16", n_pages=10, max_pages=20)
    c = s.call
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    s.step([80, 60], [80, 60])  # 5 + 4 pages
    c.plan(i32([0, 40, 41]), i32([120, 61]))
    assert int(c.status) == fl.ERR_NO_PAGES and c.held_len.tolist() == [80, 60] and int(c.n_free) == 1
    assert (c.slot_map == -1).all()
    s.step([0, 1], [0, 61])  # request 0 ends instead
    s.pages_are_whole([0, 61])
    s.step([96, 1], [96, 62])  # 6 + 4 pages
    s.pages_are_whole([96, 62])


def test_random_serving():
    rng = random.Random(5)
    s = Server(5, 120, "e4m3", n_pages=40, max_pages=12, layers=1, seed=9)
    lens = [0] * 5
    for _ in range(12):
        q_len, kv_len, left = [], [], 120
        for r in range(5):
            kind = rng.choice(["decode", "chunk", "end", "back", "idle"])
            n = min(left, {"decode": 1, "chunk": rng.randrange(1, 40), "end": 0, "back": 3, "idle": 0}[kind])
            kv = 0 if kind == "end" else max(0, lens[r] - (rng.randrange(0, 30) if kind == "back" else 0)) + n
            if kv > 150:
                n, kv = 0, 0
            q_len.append(n)
            kv_len.append(kv)
            left -= n
        if sum(-(-n // 16) for n in kv_len) > 40:
            q_len, kv_len = [0] * 5, [0] * 5
        s.step(q_len, kv_len)
        s.pages_are_whole(kv_len)
        lens = kv_len
