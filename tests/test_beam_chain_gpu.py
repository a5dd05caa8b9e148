"""GPU: the calls of a beam search together, as a decode loop makes them.

Prompts go through extension and append into an empty pool; then, step by step, the
tables follow the beams' parents, one token a beam is appended, the beams are decoded,
their logits selected from and their histories reordered.  What a beam's table names is
compared, byte for byte, with a pool into which the beam's history is appended by
itself, its decode bit for bit with that pool's, and its selection with float64.
"""
import pytest
import torch

from split_kv_mla_gb300 import mla

from test_beam_gpu import check as check_selection
from test_beam_gpu import exact_scores

pytestmark = pytest.mark.gpu

W, H, V, END, STEPS, ROWS = 3, 16, 301, 7, 12, 3000
PROMPTS = [37, 130]
B = len(PROMPTS)
CAP = W * (sum(PROMPTS) + B * (STEPS + 1))
KV_SCALE = 1.0 / 32.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    mla.load()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


class Loop:
    """A model of one layer: a token's row, query and output weights are drawn."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.kv = torch.randn(V, 576, generator=g).to(torch.bfloat16).cuda()
        self.q = torch.randn(V, H, 576, generator=g).to(torch.bfloat16).cuda()
        self.out = (torch.randn(H * 512, V, generator=g) * 0.15).cuda()
        ang = torch.rand(400, 32, generator=g) * 6.28
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).cuda()
        self.prompts = torch.randint(8, V, (sum(PROMPTS),), generator=g).int().cuda()
        self.pool = torch.zeros(ROWS, 576, dtype=torch.uint8, device="cuda")
        self.free = torch.randperm(ROWS, generator=g).int().cuda()
        self.cursor = i32(1)
        self.ws = mla.cache_workspace(ROWS)
        self.bws = mla.beam_workspace(B, W, V)
        self.plan = mla.mla_decode_plan(B * W, 1, H, CAP, mla.sm_count())
        self.dws = mla.workspace(self.plan)

    def append(self, tokens, slots, positions):
        t = tokens.long()
        return mla.mla_cache_append(self.kv[t], slots, self.pool, positions, self.cos_sin, KV_SCALE,
                                    q=self.q[t], kv_norm_cols=512, workspace_t=self.ws)

    def decode(self, q, table, indptr, lens, pool=None):
        return mla.mla_decode(self.plan, *q, self.pool if pool is None else pool, lens, table,
                              indptr, 576 ** -0.5, KV_SCALE, workspace_t=self.dws)[0]

    def logits(self, o):
        return torch.matmul(o.float().view(-1, H * 512), self.out)

    def prefill(self):
        """Tables of B requests, and what the first selection needs."""
        n = torch.tensor(PROMPTS, dtype=torch.int32, device="cuda")
        table, indptr, lens, slots, positions, tokptr, _ = mla.mla_cache_extend(
            i32(0), i32(B + 1), i32(B), self.cursor, sum(PROMPTS), sum(PROMPTS), ROWS, new_tokens=n,
            free_slots=self.free, new_cursor=self.cursor, workspace_t=self.ws)
        q = self.append(self.prompts, slots, positions)
        last = (tokptr[1:] - 1).long()
        plan = mla.mla_decode_plan(B, 1, H, sum(PROMPTS), mla.sm_count())
        o = mla.mla_decode(plan, *(t[last] for t in q), self.pool, lens, table, indptr, 576 ** -0.5,
                           KV_SCALE)[0]
        # every beam of a request sees its row; the first alone is one
        self.scores = torch.full((B, W), -torch.inf, device="cuda")
        self.scores[:, 0] = 0
        self.done = torch.zeros(B, W, dtype=torch.bool, device="cuda")
        self.x = self.logits(o).repeat_interleave(W, 0)
        # the beams' buffers, two of each
        self.tables = [[i32(CAP), i32(B * W + 1), i32(B * W)] for _ in range(2)]
        self.hist = [[i32(B * W, 400), i32(B * W)] for _ in range(2)]
        for k, t in enumerate((table, indptr, lens)):
            self.tables[0][k][:t.numel()] = t
        start = 0
        for b, m in enumerate(PROMPTS):
            self.hist[0][0][b, :m] = self.prompts[start:start + m]
            self.hist[0][1][b] = m
            start += m
        # (as many rows as beams: those of the requests first)
        self.tables[0][1][B + 1:] = self.tables[0][1][B]

    def select(self):
        self.tokens, self.parents, _, _ = mla.mla_beam_select(
            self.x, self.scores, finished=self.done, end_token=END, scores_out=self.scores,
            finished_out=self.done, workspace_t=self.bws)

    def advance(self, k, parents):
        """From buffers k to the others: histories, tables, the new rows, the logits."""
        (h0, n0), (h1, n1) = self.hist[k], self.hist[1 - k]
        tokens = self.tokens.view(-1)
        mla.mla_beam_reorder(h0, parents, n0, tokens, h1, n1, workspace_t=self.ws)
        t1 = self.tables[1 - k]
        table, indptr, lens, slots, positions, _, _ = mla.mla_cache_extend(
            *self.tables[k], self.cursor, CAP, B * W, ROWS, parents=parents, free_slots=self.free,
            table=t1[0], indptr=t1[1], lens=t1[2], new_cursor=self.cursor, workspace_t=self.ws)
        q = self.append(tokens, slots, positions)
        self.o = self.decode(q, table, indptr, lens)
        self.x = self.logits(self.o)

    def compact(self, k):
        """Live rows to the front; the free slots are then what follows, in order."""
        n = int(self.tables[k][1][-1])
        table, live = mla.mla_cache_compact(self.pool, self.tables[k][0][:n].clone(),
                                            workspace_t=self.ws)
        self.tables[k][0][:n] = table
        self.free.copy_(torch.arange(ROWS, device="cuda"))
        self.cursor.copy_(live)

    def check(self, k):
        table, indptr, lens = self.tables[k]
        hist, n = self.hist[k]
        assert torch.equal(n, lens) and torch.equal(indptr.diff(), lens)
        pool, q = torch.zeros(CAP, 576, dtype=torch.uint8, device="cuda"), []
        start = 0
        for f in range(B * W):
            m = int(n[f])
            t = hist[f, :m].long()
            at = torch.arange(m, dtype=torch.int32, device="cuda")
            qn, qp = mla.mla_cache_append(self.kv[t], at + start, pool, at, self.cos_sin, KV_SCALE,
                                          q=self.q[t], kv_norm_cols=512)
            q.append((qn[-1], qp[-1]))
            rows = table[int(indptr[f]):int(indptr[f + 1])].long()
            assert torch.equal(self.pool[rows], pool[start:start + m]), f
            start += m
        own = torch.arange(CAP, dtype=torch.int32, device="cuda")
        o = self.decode([torch.stack(z) for z in zip(*q)], own, indptr, lens, pool)
        assert torch.equal(o, self.o)


def first_parents(loop):
    return (loop.parents.view(-1) // W).int()


@pytest.mark.parametrize("seed", range(3))
def test_a_search(seed):
    loop = Loop(seed)
    loop.prefill()
    k, most = 0, 0
    for step in range(STEPS):
        x, s, d = loop.x.clone(), loop.scores.clone(), loop.done.clone()
        loop.select()
        check_selection((loop.tokens, loop.parents, loop.scores, loop.done),
                        exact_scores(x, s, d, END), W, V, d, END)
        loop.advance(k, first_parents(loop) if step == 0 else loop.parents.view(-1))
        k = 1 - k
        loop.check(k)
        if step % 5 == 3:
            loop.compact(k)
            assert int(loop.cursor) <= int(loop.tables[k][1][-1])
            loop.check(k)
        most = max(most, int(loop.cursor))
    assert most < ROWS
    for ws in (loop.ws, loop.bws, loop.dws):
        assert mla.mla_read_device_error(ws) == 0


def test_steps_in_one_graph():
    a, b = Loop(5), Loop(5)
    for loop in (a, b):
        loop.prefill()
        loop.select()
        loop.advance(0, first_parents(loop))
    logits = b.x     # the captured steps read and write one buffer
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for k in (1, 0):
            b.select()
            b.advance(k, b.parents.view(-1))
            logits.copy_(b.x)
            b.x = logits
    for _ in range(STEPS // 2):
        for k in (1, 0):
            a.select()
            a.advance(k, a.parents.view(-1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.hist[1][0], b.hist[1][0]) and torch.equal(a.scores, b.scores)
        assert torch.equal(a.o, b.o) and torch.equal(a.done, b.done)
        for s, t in zip(a.tables[1], b.tables[1]):
            assert torch.equal(s, t)
    for loop in (a, b):
        for ws in (loop.ws, loop.bws, loop.dws):
            assert mla.mla_read_device_error(ws) == 0
