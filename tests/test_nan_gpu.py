"""GPU: a NaN reaches the rows that see it, as NaN in o and in the LSE, and no others.

NaN e4m3fn codes in the rows that a page table names, and NaN or infinite queries,
through every way that a key takes: the split kernel with one split and several,
its reduce and its fused merge, and a shared prefix's requests' own keys both in the
prefix's tiles and in the split kernel.  Rows that do not see the NaN keep every bit.
"""
import dataclasses

import pytest
import torch

from oracle import oracle
from split_kv_mla_gb300 import inputs as gen
from split_kv_mla_gb300 import mla

from gpu_util import run_dense, run_sparse
from test_prefix_gpu import Shared, both, make, plan_of, run, variant

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    oracle.build()
    mla.load()


def plans(s):
    """The own keys in the tiles, and in the split kernel as one split and as several."""
    out = []
    for p in both(s):
        if p.joined:
            out.append(p)
            continue
        for ns in (1, 3):
            q = mla.mla_prefix_plan_t.from_buffer_copy(p)
            q.own = mla.mla_plan_force_splits(p.own, ns)
            out.append(variant(q))
    return out


def with_pool(s, pool):
    return Shared(dataclasses.replace(s.own, pool=pool), s.joined, s.prefix)


def rows_of(out, want, seen):
    """`seen` [R] rows are NaN in both outputs, the others are `want`'s bits."""
    seen = seen.cuda()
    for got, ref in zip(out, want):
        got, ref = got.reshape(seen.numel(), -1), ref.reshape(seen.numel(), -1)
        assert bool(torch.isnan(got[seen]).all())
        assert torch.equal(got[~seen], ref[~seen])
        assert not bool(torch.isnan(got[~seen]).any())


@pytest.mark.parametrize("byte", [0x7F, 0xFF])
@pytest.mark.parametrize("column", [0, 300, 511, 570])
def test_own_row_on_every_plan(byte, column):
    s = make(1, 16, 400, [30, 5, 260, 2, 9], seed=24)
    pool = s.own.pool.clone()
    pool[int(s.own.kv_indices[35 + 200]), 0, column] = byte   # the third request's
    for plan in plans(s):
        want, _ = run(s, plan)
        got, ws = run(with_pool(s, pool), plan)
        rows_of(got, want, torch.arange(5 * 16) // 16 == 2)
        assert mla.mla_read_device_error(ws) == 0


@pytest.mark.parametrize("heads", [4, 16, 24])
def test_own_row_that_only_the_last_draft_sees(heads):
    s = make(3, heads, 200, [7, 150, 40], seed=31)
    pool = s.own.pool.clone()
    pool[int(s.own.kv_indices[156]), 0, 77] = 0x7F   # the second request's last
    seen = torch.zeros(9, heads, dtype=torch.bool)
    seen[5] = True
    for plan in plans(s):
        want, _ = run(s, plan)
        got, _ = run(with_pool(s, pool), plan)
        rows_of(got, want, seen.reshape(-1))


def test_a_row_of_nan_keys_alone():
    # no prefix position in use, one own key, and it holds a NaN
    s = make(1, 16, 130, [1, 3], seed=32)
    pool = s.own.pool.clone()
    pool[int(s.own.kv_indices[0]), 0, 5] = 0x7F
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    for plan in plans(s):
        want, _ = run(s, plan, prefix_len=none)
        got, _ = run(with_pool(s, pool), plan, prefix_len=none)
        rows_of(got, want, torch.arange(32) < 16)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("prefix", [0, 200])
def test_queries_on_every_plan(value, prefix):
    s = make(1, 16, prefix, [30, 5, 260], seed=33)
    own = s.own
    seen = torch.zeros(3, 16, dtype=torch.bool)
    lat, pe = own.q_lat.clone(), own.q_pe.clone()
    for b, h, t, c in ((0, 0, lat, 3), (1, 7, pe, 63), (2, 15, lat, 511)):
        t[b, h, c] = value
        seen[b, h] = True
    for plan in plans(s):
        want, _ = run(s, plan)
        got, _ = run(Shared(dataclasses.replace(own, q_lat=lat, q_pe=pe), s.joined, s.prefix),
                     plan)
        rows_of(got, want, seen.reshape(-1))


@pytest.mark.parametrize("ns,mc", [(1, 1), (2, 1), (8, 1), (20, 1), (4, 4), (8, 2)])
@pytest.mark.parametrize("q_len,heads", [(1, 16), (4, 16), (1, 5)])
def test_decode(ns, mc, q_len, heads):
    inp = gen.dense_inputs(3, q_len, heads, [700, 2600, 90], seed=40 + ns)
    plan = mla.mla_plan_force_splits(
        mla.mla_decode_plan(3, q_len, heads, inp.total_keys, mla.sm_count()), ns)
    plan.merge_cluster = mc
    want = run_dense(inp, plan)[:2]
    at = int(inp.kv_indptr[1]) + 2600 - 2   # seen by the second request's last two drafts
    pool = inp.pool.clone()
    pool[int(inp.kv_indices[at]), 0, 130] = 0xFF
    got = run_dense(dataclasses.replace(inp, pool=pool), plan)[:2]
    t = torch.arange(3 * q_len)
    seen = (t // q_len == 1) & (t % q_len >= q_len - 2)
    rows_of(got, want, seen[:, None].expand(-1, heads).reshape(-1))


def test_stage_reused_by_a_short_block():
    # draft rows that see neither the NaN nor the last, short block, which reuses the
    # stage of the block that held it
    inp = gen.dense_inputs(1, 300, 1, [517], seed=50)
    pool = inp.pool.clone()
    pool[int(inp.kv_indices[356]), 0, 9] = 0x7F   # block 2 of 5; row t sees 217 + t
    base = mla.mla_decode_plan(1, 300, 1, 517, mla.sm_count())
    plan = mla.mla_plan_force_splits(base, 1)
    want = run_dense(inp, plan)[:2]
    got = run_dense(dataclasses.replace(inp, pool=pool), plan)[:2]
    rows_of(got, want, torch.arange(300) + 217 >= 356)


def test_sparse_and_second_cache():
    inp = gen.sparse_inputs(3, 16, 300, pool_rows=4000, seed=60)
    pool = inp.pool.clone()
    slot = int(inp.indices[1, 250])
    pool[slot].view(-1)[460] = 0x7F   # RoPE part of a 512-byte row
    seen = (inp.indices == slot).any(1)
    assert bool(seen[1]) and not bool(seen.all())
    for splits in (1, 2):
        plan = mla.mla_sparse_decode_plan(3, 16, 300, mla.sm_count(), splits)
        want = run_sparse(inp, plan)[:2]
        got = run_sparse(dataclasses.replace(inp, pool=pool), plan)[:2]
        rows_of(got, want, seen[:, None].expand(-1, 16).reshape(-1))


def test_shares_of_nan_in_the_merges():
    # a NaN LSE among the partials, and beside partials that saw no key
    lse = torch.tensor([[1.0, float("nan")], [-float("inf"), float("nan")], [0.5, 2.0],
                        [-float("inf")] * 2], device="cuda")
    o = torch.ones(4, 2, 512, device="cuda")
    got, gl = mla.mla_splitk_reduce(o, lse)
    rows_of((got, gl), (got.nan_to_num(), gl), torch.tensor([True, True, False, False]))
    assert bool((got[3] == 0).all()) and float(gl[3]) == -float("inf")
    got, gl = mla.mla_dcp_lse_merge_ranks(o.transpose(0, 1).contiguous(), lse.t().contiguous())
    rows_of((got, gl), (got.nan_to_num(), gl), torch.tensor([True, True, False, False]))
    assert bool((got[3] == 0).all()) and float(gl[3]) == -float("inf")
