"""GPU: query rows with one column far above the others, which the keys do not answer
to, so that the logits are made of the small columns alone.

Two e4m3 terms carry a query's element to 2^-23 of the row's largest one at best; with
a column 2^14 (2^16) times the others and zero in the keys, that is up to 0.010 (0.047)
nats on a logit over 500 rows and 2000 keys (emulated on the CPU with the types'
roundings), past the bar of 1e-3 on the LSE.  With the third term, in e5m2, it is up to
1.5e-4 (1.2e-3); the LSE averages that over its keys.
"""
import dataclasses

import pytest
import torch

from oracle import oracle
from split_kv_mla_gb300 import inputs as gen
from split_kv_mla_gb300 import mla

from test_prefix_gpu import both, check, join, make, plan_of, run, variant, wait_runs_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    oracle.build()
    mla.load()


def silent_outlier(s, ratio, part="lat", rows=None):
    """One column of the rows' queries (all of them, or the (row, head) pairs of `rows`) is
    `ratio` and zero in every key."""
    own = s.own
    col = 77 if part == "lat" else 512 + 13
    lat, pe = own.q_lat.clone(), own.q_pe.clone()
    t = lat if part == "lat" else pe
    c = col if part == "lat" else col - 512
    for r, h in ([(slice(None), slice(None))] if rows is None else rows):
        t[r, h, c] = ratio
    pool = own.pool.clone()
    pool.view(-1, 576)[:, col] = 0
    return join(dataclasses.replace(own, q_lat=lat, q_pe=pe, pool=pool), s.prefix)


@pytest.mark.parametrize("part", ["lat", "pe"])
@pytest.mark.parametrize("power", [9, 12, 14, 16])
def test_outlier_that_the_keys_do_not_answer_to(power, part):
    s = silent_outlier(make(1, 16, 900, [60, 700], seed=12), 2.0 ** power, part)
    for plan in both(s):
        check(s, f"2^{power} {part} joined {plan.joined}", plan=plan)


def test_as_the_joined_decode():
    s = silent_outlier(make(2, 16, 1500, [260, 9, 40], seed=13), 2.0 ** 14)
    j = s.joined
    plan = mla.mla_decode_plan(j.batch, 2, 16, j.total_keys, mla.sm_count())
    _, want = mla.mla_decode(plan, j.q_lat.cuda(), j.q_pe.cuda(), j.pool.cuda(),
                             j.seq_lens.cuda(), j.kv_indices.cuda(), j.kv_indptr.cuda(), j.scale,
                             j.kv_scale)
    for p in both(s):
        (_, lse), _ = run(s, p)
        # 1.5e-4 nats at most from this call's terms, 7.5e-5 from the other's, in base 2;
        # and 1e-4 for both calls' exponentials, logarithms and fp32 sums
        assert float((lse - want).abs().max()) <= (1.5e-4 + 7.5e-5) * 1.4427 + 1e-4


@pytest.mark.parametrize("ctas,splits", [(1, 0), (2, 0), (3, 0), (7, 0), (40, 0), (None, 1),
                                         (None, 3), (None, 9)])
def test_tiles_with_and_without_a_third_term_in_one_cta(ctas, splits):
    # nine tiles, the fourth, fifth and last with such rows: a CTA's runs change between
    # the two ways of a tile, at odd and even block counts
    s = make(1, 24, 900, [5, 300, 17, 64, 9, 1, 80, 33, 2, 0, 130, 3, 7, 7, 7, 1, 2, 60, 8, 4, 3,
                          9, 5, 2], seed=24)
    rows = [(9, 3), (10, 23), (23, 23)]   # tiles 3, 4 (rows 219 and 263 of 576) and 8
    for part in ("lat", "pe"):
        loud = silent_outlier(s, 2.0 ** 14, part, rows)
        quiet = silent_outlier(s, 0.0, part, rows)
        for joined in (0, 1):
            plan = variant(plan_of(s), joined=joined, ctas=ctas or 9 * splits, splits=splits)
            o, lse = check(loud, f"{part} joined {joined}", plan=plan)
            (o2, lse2), _ = run(quiet, plan)
            tile = torch.arange(576) // 64
            same = (tile != 3) & (tile != 4) & (tile != 8)
            same = same.cuda()
            assert torch.equal(o.view(576, 512)[same], o2.view(576, 512)[same])
            assert torch.equal(lse.view(-1)[same], lse2.view(-1)[same])
            if joined:   # nor do such a tile's other rows change
                same = torch.ones(576, dtype=torch.bool, device="cuda")
                same[[r * 24 + h for r, h in rows]] = False
                assert torch.equal(o.view(576, 512)[same], o2.view(576, 512)[same])
                assert torch.equal(lse.view(-1)[same], lse2.view(-1)[same])


def test_repeat_and_long_runs():
    s = silent_outlier(make(1, 64, 9000, [100, 3], seed=25), 2.0 ** 13)
    plan = variant(plan_of(s), joined=1, ctas=2, splits=1)
    ws = mla.workspace(plan)
    o, lse = check(s, "71 blocks a run", plan=plan, ws=ws)
    (o2, lse2), _ = run(s, plan, ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_wait_that_runs_out_in_such_a_tile():
    s = silent_outlier(make(1, 64, 1000, [30, 5], seed=20), 2.0 ** 14)
    for plan in both(s) + [variant(plan_of(s), ctas=1, splits=0, joined=1)]:
        wait_runs_out(s, plan)
