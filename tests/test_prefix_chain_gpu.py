"""GPU: the cache and shared-prefix operators together, as a serving loop uses
them: a prompt is appended, forked, decoded with its rows shared, its requests
grow, end, and the pool is compacted; every decode against the fp64 oracle on
the rows that a plain float64 append gives.

The oracle reads the pool's own bytes, so the append is checked by itself
(test_cache_gpu.py's tolerance) and the decodes by the parity bar.
"""
import numpy as np
import pytest
import torch

from oracle import oracle
from split_kv_mla_gb300 import inputs as gen
from split_kv_mla_gb300 import mla

from gpu_util import compare
from test_cache_gpu import check_bf16, check_e4m3, normed, rotate

pytestmark = pytest.mark.gpu

H, W, SCALE, KV_SCALE, EPS = 16, 576, 576 ** -0.5, 1.0 / 32, 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    oracle.build()
    mla.load()


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


class Loop:
    """The pool, its free slots and the tables of the requests that are alive."""

    def __init__(self, rows, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.pool = torch.zeros(rows, W, dtype=torch.uint8, device="cuda")
        self.free = torch.randperm(rows, generator=self.g).tolist()
        ang = torch.rand(4096, 32, generator=self.g, dtype=torch.float64) * 6.28
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
        self.weight = (1 + 0.1 * torch.randn(512, generator=self.g)).to(torch.bfloat16)
        self.ws = mla.cache_workspace(rows)
        self.tables = []

    def take(self, n):
        out, self.free = self.free[:n], self.free[n:]
        return out

    def append(self, positions, slots):
        """Rows and queries of new tokens; returns the absorbed query's parts."""
        T = len(positions)
        kv = (torch.randn(T, W, generator=self.g) * 2).to(torch.bfloat16)
        q = torch.randn(T, H, 192, generator=self.g).to(torch.bfloat16)
        _, q_pe = mla.mla_cache_append(
            kv.cuda(), i32(slots), self.pool, i32(positions), self.cos_sin.cuda(), KV_SCALE,
            q=q.cuda(), kv_weight=self.weight.cuda(), kv_norm_cols=512, eps=EPS,
            workspace_t=self.ws)
        cs = self.cos_sin.double()[torch.tensor(positions)]
        x = normed(kv.double(), 512, self.weight, EPS)
        size = x.abs()
        x[:, 512:], size[:, 512:] = rotate(x[:, 512:], cs[:, :32], cs[:, 32:], False)
        check_e4m3(self.pool[torch.tensor(slots).cuda()], x / KV_SCALE, size / KV_SCALE)
        want, qs = rotate(q.double()[..., 128:], cs[:, None, :32], cs[:, None, 32:], False)
        check_bf16(q_pe, want, qs)
        q_lat = torch.randn(T, H, 512, generator=self.g).to(torch.bfloat16)
        return q_lat, q_pe

    def decode(self, q_lat, q_pe, shared):
        """The requests' next token: `shared` first slots are the same in every table."""
        B = len(self.tables)
        own = [t[shared:] for t in self.tables]
        ptr = i32(np.cumsum([0] + [len(t) for t in own]))
        total = sum(map(len, own))
        plan = mla.mla_prefix_decode_plan(B, 1, H, shared, total, mla.sm_count())
        ws = mla.workspace(plan)
        o, lse = mla.mla_prefix_decode(
            plan, q_lat.cuda(), q_pe, self.pool, i32(self.tables[0][:shared]),
            i32([len(t) for t in own]), i32(sum(own, [])), ptr, SCALE, KV_SCALE, workspace_t=ws)
        torch.cuda.synchronize()
        joined = gen.DenseInputs(
            batch=B, q_len=1, num_heads=H, q_lat=q_lat, q_pe=q_pe.cpu(),
            pool=self.pool.cpu().view(-1, 1, W),
            seq_lens=torch.tensor([len(t) for t in self.tables]).int(),
            kv_indices=torch.tensor(sum(self.tables, [])).int(),
            kv_indptr=torch.tensor(np.cumsum([0] + [len(t) for t in self.tables])).int(),
            scale=SCALE, kv_scale=KV_SCALE)
        ro, rl = oracle.dense_decode(joined)
        compare(o, lse, ro, rl, f"{B} requests, {shared} shared")
        assert mla.mla_read_device_error(ws) == 0
        # the plain decode on the joined tables gives the same
        p2 = mla.mla_decode_plan(B, 1, H, joined.total_keys, mla.sm_count())
        o2, _ = mla.mla_decode(p2, q_lat.cuda(), q_pe, self.pool, joined.seq_lens.cuda(),
                               joined.kv_indices.cuda(), joined.kv_indptr.cuda(), SCALE, KV_SCALE)
        compare(o2, lse, ro, rl, "plain decode")
        return o


def test_a_prompt_appended_forked_decoded_and_compacted():
    loop = Loop(4000, seed=1)
    P, F = 1300, 6
    prompt = loop.take(P)
    for c in range(0, P, 500):   # prefill in chunks
        loop.append(list(range(c, min(P, c + 500))), prompt[c:c + 500])
    # six samples that share 1290 positions and own a copy of the last ten
    keep = 1290
    fresh = loop.take(F * (P - keep))
    table = mla.mla_cache_fork(
        loop.pool, i32(prompt), i32([0, P]), i32([0] * F), i32([keep] * F),
        i32([P * f for f in range(F + 1)]), P * F, i32(fresh),
        i32([(P - keep) * f for f in range(F + 1)]), workspace_t=loop.ws)
    loop.tables = table.cpu().view(F, P).tolist()
    assert all(t[:keep] == prompt[:keep] for t in loop.tables)
    assert len({s for t in loop.tables for s in t[keep:]}) == F * (P - keep)
    for step in range(4):   # every request appends a token and attends
        slots = loop.take(F)
        q_lat, q_pe = loop.append([P + step] * F, slots)
        for t, s in zip(loop.tables, slots):
            t.append(s)
        loop.decode(q_lat, q_pe, keep)
    # two requests end; the live rows move to the front
    loop.tables = [loop.tables[i] for i in (0, 2, 3, 5)]
    before = loop.pool[torch.tensor(sum(loop.tables, [])).cuda()].clone()
    new, live = mla.mla_cache_compact(loop.pool, i32(sum(loop.tables, [])), workspace_t=loop.ws)
    assert torch.equal(loop.pool[new.long()], before)
    live = int(live)
    assert live == len(set(sum(loop.tables, []))) and int(new.max()) == live - 1
    n = len(loop.tables[0])
    loop.tables = new.cpu().view(4, n).tolist()
    loop.free = list(range(live, 4000))
    slots = loop.take(4)
    q_lat, q_pe = loop.append([P + 4] * 4, slots)
    for t, s in zip(loop.tables, slots):
        t.append(s)
    loop.decode(q_lat, q_pe, keep)
    assert mla.mla_read_device_error(loop.ws) == 0


def test_one_step_in_one_graph():
    # append and decode of the next token captured together and replayed on new inputs
    loop = Loop(2000, seed=2)
    P, B = 700, 3
    prompt = loop.take(P)
    loop.append(list(range(P)), prompt)
    own = [loop.take(5) for _ in range(B)]
    for j in range(4):
        loop.append([P + j] * B, [t[j] for t in own])
    g = loop.g
    kv = torch.randn(B, W, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(B, H, 64, generator=g).to(torch.bfloat16).cuda()
    q_lat = torch.randn(B, H, 512, generator=g).to(torch.bfloat16).cuda()
    slots, pos, cs = i32([t[4] for t in own]), i32([P + 4] * B), loop.cos_sin.cuda()
    prefix, lens = i32(prompt), i32([5] * B)
    idx, ptr = i32(sum(own, [])), i32([0, 5, 10, 15])
    w, plan = loop.weight.cuda(), mla.mla_prefix_decode_plan(B, 1, H, P, 15, mla.sm_count())
    ws = mla.workspace(plan)

    def step():
        _, q_pe = mla.mla_cache_append(kv, slots, loop.pool, pos, cs, KV_SCALE, q=q, kv_weight=w,
                                       kv_norm_cols=512, workspace_t=loop.ws)
        return q_pe, mla.mla_prefix_decode(plan, q_lat, q_pe, loop.pool, prefix, lens, idx, ptr,
                                           SCALE, KV_SCALE, workspace_t=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q_pe, (o, lse) = step()
    for _ in range(3):
        kv.copy_(torch.randn(B, W, generator=g))
        q.copy_(torch.randn(B, H, 64, generator=g))
        q_lat.copy_(torch.randn(B, H, 512, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        joined = gen.DenseInputs(
            batch=B, q_len=1, num_heads=H, q_lat=q_lat.cpu(), q_pe=q_pe.cpu(),
            pool=loop.pool.cpu().view(-1, 1, W), seq_lens=torch.tensor([P + 5] * B).int(),
            kv_indices=torch.cat([torch.tensor(prompt + t) for t in own]).int(),
            kv_indptr=torch.arange(B + 1).int() * (P + 5), scale=SCALE, kv_scale=KV_SCALE)
        ro, rl = oracle.dense_decode(joined)
        compare(o, lse, ro, rl, "graph")
    assert mla.mla_read_device_error(ws) == 0 and mla.mla_read_device_error(loop.ws) == 0
