"""GPU: decode over a shared prefix against the fp64 oracle on the joined page
tables, with the framework's parity bar (gpu_util.compare).

The bar holds by the number formats: a probability is an e4m3 term plus an e5m2
term, off by at most 2^-4 2^-3 = 2^-7 of itself and 0.0014 in the mean square,
normalised by the sum of what was fed, on top of the output's own bf16 rounding
(2^-8 at most, 0.0017 in the mean square): about 0.0022 relative RMS against a
bar of 0.005.  Logits carry the bf16 queries to 2^-23 of a row's largest element.
"""
import dataclasses

import numpy as np
import pytest
import torch

from oracle import oracle
from split_kv_mla_gb300 import inputs as gen
from split_kv_mla_gb300 import mla

from gpu_util import compare
from test_prefix_host import workspace_bytes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    oracle.build()
    mla.load()


@dataclasses.dataclass
class Shared:
    own: gen.DenseInputs        # the requests' own keys
    joined: gen.DenseInputs     # the same requests with the prefix in front
    prefix: torch.Tensor        # int32 [P]


def join(own, prefix):
    P = prefix.numel()
    lens, at, parts = own.seq_lens.long(), own.kv_indptr.long(), []
    for b in range(own.batch):
        parts += [prefix, own.kv_indices[at[b]:at[b] + lens[b]]]
    ptr = torch.zeros(own.batch + 1, dtype=torch.int64)
    ptr[1:] = torch.cumsum(lens + P, 0)
    return Shared(own, dataclasses.replace(
        own, seq_lens=(lens + P).int(), kv_indices=torch.cat(parts).int(), kv_indptr=ptr.int()),
        prefix.int())


def make(q_len, heads, P, lens, seed, **kw):
    own = gen.dense_inputs(len(lens), q_len, heads, lens, seed, extra_slots=P + 37, **kw)
    free = np.setdiff1d(np.arange(own.pool.shape[0]), own.kv_indices.numpy())
    pick = np.random.default_rng(seed).permutation(free)[:P]
    return join(own, torch.from_numpy(pick.astype(np.int32)))


def to_cuda(s):
    o = s.own
    return dict(q_lat=o.q_lat.cuda(), q_pe=o.q_pe.cuda(), pool=o.pool.cuda(),
                prefix_indices=s.prefix.cuda(), seq_lens=o.seq_lens.cuda(),
                kv_indices=o.kv_indices.cuda(), kv_indptr=o.kv_indptr.cuda())


def plan_of(s, cap=None, sms=None):
    o = s.own
    return mla.mla_prefix_decode_plan(o.batch, o.q_len, o.num_heads,
                                      s.prefix.numel() if cap is None else cap, o.total_keys,
                                      sms or mla.sm_count())


def variant(plan, **fields):
    """The plan with other launch choices."""
    p = mla.mla_prefix_plan_t.from_buffer_copy(plan)
    for k, v in fields.items():
        setattr(p, k, v)
    p.workspace_bytes = workspace_bytes(p)
    return p


def both(s):
    """The plan with the requests' own keys in the tiles, and in the split kernel."""
    plan = plan_of(s)
    return [variant(plan, joined=j) for j in ((0, 1) if s.own.total_keys and plan.ctas else (0,))]


def run(s, plan=None, ws=None, d=None, **kw):
    d = d or to_cuda(s)
    plan = plan or plan_of(s)
    ws = mla.workspace(plan) if ws is None else ws
    out = mla.mla_prefix_decode(plan, **d, scale=s.own.scale, kv_scale=s.own.kv_scale,
                                workspace_t=ws, **kw)
    torch.cuda.synchronize()
    return out, ws


def check(s, what="", errors=0, **kw):
    (o, lse), ws = run(s, **kw)
    ro, rl = oracle.dense_decode(s.joined)
    compare(o, lse, ro, rl, what)
    assert mla.mla_read_device_error(ws) == errors
    return o, lse


@pytest.mark.parametrize("q_len,heads,P,lens", [
    (1, 1, 1, [0]), (1, 1, 1, [1]), (1, 16, 128, [3]), (1, 16, 127, [1, 0, 5]),
    (1, 16, 129, [200, 1]), (1, 64, 256, [0, 0]), (1, 128, 640, [7, 130]),
    (1, 5, 1000, [33, 0, 1, 129, 64]), (2, 16, 300, [2, 9]), (4, 16, 2001, [4, 70, 500]),
    (7, 3, 131, [7, 8]), (1, 16, 5000, [600] * 9), (1, 128, 4096, [17, 400, 3, 90]),
    (1, 33, 8192, [50] * 20), (8, 128, 700, [11, 40])])
def test_prefix(q_len, heads, P, lens):
    s = make(q_len, heads, P, lens, seed=P + heads)
    for plan in both(s):
        check(s, f"q{q_len} H{heads} P{P} joined {plan.joined}", plan=plan)


@pytest.mark.parametrize("heads,lens", [
    (1, [3, 0, 0, 200, 1, 0, 129] * 11), (2, [5] * 33), (24, [5, 300, 17, 64, 9, 1, 80, 33, 2]),
    (24, [0, 0, 0, 0, 0]), (128, [1, 128, 129, 0, 700]), (65, [50, 60, 70]), (96, [300, 2])])
@pytest.mark.parametrize("ctas,splits", [(1, 0), (2, 0), (3, 0), (5, 0), (11, 0), (37, 0),
                                         (152, 0), (None, 1), (None, 2), (None, 13)])
def test_any_cut_of_the_blocks(heads, lens, ctas, splits):
    # runs that end inside tiles, several tiles per CTA, CTAs of one block or none,
    # tiles of many requests and requests of several tiles
    s = make(1, heads, 500, lens, seed=heads)
    plan = plan_of(s)
    ctas = ctas or plan.tiles * splits
    for joined in (0, 1) if s.own.total_keys else (0,):
        check(s, f"{ctas} CTAs, {splits} splits, joined {joined}",
              plan=variant(plan, ctas=ctas, splits=splits, joined=joined))


def test_one_request_far_longer_than_the_others():
    s = make(1, 16, 600, [3, 5000, 0, 40, 7, 1, 1, 900], seed=21)
    for plan in both(s):
        check(s, f"skewed, joined {plan.joined}", plan=plan)
        check(s, f"skewed, joined {plan.joined}", plan=variant(plan, ctas=152, splits=0))


def test_tables_with_room_to_spare():
    # a table longer than its request's length, starting past entry 0
    s = make(2, 16, 300, [30, 0, 150], seed=22)
    own = s.own
    lens, ptr = own.seq_lens, own.kv_indptr
    new_ptr = torch.tensor([7, 7 + 200, 7 + 203, 7 + 203 + 150]).int()
    idx = torch.full((int(new_ptr[-1]),), 2 ** 30, dtype=torch.int32)
    for b in range(3):
        idx[int(new_ptr[b]):int(new_ptr[b]) + int(lens[b])] = \
            own.kv_indices[int(ptr[b]):int(ptr[b]) + int(lens[b])]
    d = to_cuda(s)
    d.update(kv_indices=idx.cuda(), kv_indptr=new_ptr.cuda())
    base = mla.mla_prefix_decode_plan(3, 2, 16, 300, idx.numel(), mla.sm_count())
    for joined in (0, 1):
        check(s, f"spare, joined {joined}", plan=variant(base, joined=joined), d=d)


def test_bad_lengths_are_clamped_and_reported():
    s = make(1, 16, 300, [30, 20, 150], seed=23)
    for joined in (0, 1):
        plan = variant(plan_of(s), joined=joined)
        d = to_cuda(s)
        d["seq_lens"] = torch.tensor([30, 21, -4], dtype=torch.int32, device="cuda")
        (o, lse), ws = run(s, plan, d=d)
        assert mla.mla_read_device_error(ws) == mla.MLA_DEVERR_BAD_LENGTH
        cut = dataclasses.replace(s.own, seq_lens=torch.tensor([30, 20, 0]).int())
        ro, rl = oracle.dense_decode(join(cut, s.prefix).joined)
        compare(o, lse, ro, rl, f"joined {joined}")


def test_no_prefix_and_no_keys_at_all():
    s = make(1, 16, 0, [40, 0, 7], seed=1)
    o, lse = check(s, "no prefix")
    assert bool((o[1] == 0).all()) and bool((lse[1] == -float("inf")).all())
    (o, lse), _ = run(make(1, 16, 0, [0, 0], seed=2))   # (the oracle wants one key at least)
    assert bool((o == 0).all()) and bool((lse == -float("inf")).all())
    s = make(1, 16, 200, [0, 0], seed=2)
    check(s, "only the prefix")


def test_lengths_without_a_table_are_reported():
    s = make(1, 16, 200, [0, 0], seed=26)
    d = to_cuda(s)
    d["seq_lens"] = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    (o, lse), ws = run(s, d=d)
    assert mla.mla_read_device_error(ws) == mla.MLA_DEVERR_BAD_LENGTH
    ro, rl = oracle.dense_decode(s.joined)
    compare(o, lse, ro, rl, "clamped to none")


def test_length_on_the_device():
    # one plan and one captured graph serve every length up to the capacity
    s = make(2, 16, 1400, [30, 2, 250], seed=8)
    for plan in both(s):
        lengths_on_the_device(s, plan)
    lengths_on_the_device(s, variant(plan_of(s), ctas=40, splits=0))


def lengths_on_the_device(s, plan):
    d = to_cuda(s)
    ws = mla.workspace(plan)
    n = torch.tensor([1400], dtype=torch.int32, device="cuda")
    run(s, plan, ws, d, prefix_len=n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = mla.mla_prefix_decode(plan, **d, scale=s.own.scale, kv_scale=s.own.kv_scale,
                                       prefix_len=n, workspace_t=ws)
    for length in (1400, 1, 0, 127, 128, 129, 777, 1399):
        n.fill_(length)
        graph.replay()
        torch.cuda.synchronize()
        cut = join(s.own, s.prefix[:length])
        ro, rl = oracle.dense_decode(cut.joined)
        compare(o, lse, ro, rl, f"length {length}")
    assert mla.mla_read_device_error(ws) == 0
    for length, same in ((1500, 1400), (-3, 0)):
        n.fill_(length)
        graph.replay()
        assert mla.mla_read_device_error(ws) == mla.MLA_DEVERR_BAD_LENGTH
        mla.mla_workspace_reset(ws)
        cut = join(s.own, s.prefix[:same])
        ro, rl = oracle.dense_decode(cut.joined)
        compare(o, lse, ro, rl, f"clamped {length}")


def test_drafts_that_reach_back_into_the_prefix():
    # fewer own keys than draft rows: the first rows do not see the prefix's end
    s = make(4, 16, 300, [0, 1, 2, 3, 4], seed=9)
    for plan in both(s):
        check(s, "window in the prefix", plan=plan)
    s = make(6, 8, 3, [0, 1, 2], seed=10)   # rows that see nothing at all
    for plan in both(s):
        o, lse = check(s, "empty rows", plan=plan)
        assert bool((lse[0] == -float("inf")).all()) and bool((o[0] == 0).all())


def test_same_slots_twice_and_joined_decode():
    # a slot named by the prefix and by requests; the plain decode agrees
    s = make(1, 16, 700, [90, 10], seed=11)
    s.own.kv_indices[:20] = s.prefix[100:120]
    s.prefix[5:9] = s.prefix[5]
    s = join(s.own, s.prefix)
    for plan in both(s):
        o, lse = check(s, "repeated slots", plan=plan)
    j = s.joined
    plan = mla.mla_decode_plan(j.batch, 1, 16, j.total_keys, mla.sm_count())
    o2, lse2 = mla.mla_decode(plan, j.q_lat.cuda(), j.q_pe.cuda(), j.pool.cuda(),
                              j.seq_lens.cuda(), j.kv_indices.cuda(), j.kv_indptr.cuda(), j.scale,
                              j.kv_scale)
    assert float((lse - lse2).abs().max()) <= 1e-3
    assert float((o.float() - o2.float()).abs().max()) <= 2e-2


@pytest.mark.parametrize("edge", ["lat 2^8", "lat 2^12", "pe 2^10", "pe x32", "lat tiny",
                                  "sharp", "tied", "dominant", "tiny queries"])
def test_number_format_edges(edge):
    s = make(1, 16, 900, [60, 3], seed=12)
    own = s.own
    if edge.startswith("lat 2"):
        gen.plant_query_outliers(own, 2.0 ** int(edge.split("^")[1]), 5)
    elif edge.startswith("pe 2"):
        gen.plant_query_outliers(own, 2.0 ** 10, 5, "pe")
    elif edge == "pe x32":
        gen.scale_query_parts(own, pe=32.0)
    elif edge == "lat tiny":
        gen.scale_query_parts(own, lat=2.0 ** -10)
    elif edge == "sharp":
        gen.scale_query_parts(own, lat=30.0, pe=30.0)
    elif edge == "tied":
        gen.near_tied_pool(own, 6)
    elif edge == "tiny queries":
        gen.scale_query_parts(own, lat=2.0 ** -60, pe=2.0 ** -60)
    else:
        gen.share_query_across_heads(own)
        joined = join(own, s.prefix).joined
        own.pool = gen.plant_dominant_key(joined, 0.8, 7).pool
    s = join(own, s.prefix)
    for plan in both(s):
        check(s, edge, plan=plan)


@pytest.mark.parametrize("gap", [6.0, 10.0, 13.0])
def test_one_sink_key_over_many_weak_ones(gap):
    # a key `gap` nats above 20,000 others: their weights sit 9 to 19 bits below it
    s = make(1, 4, 20000, [1], seed=13)
    own = s.own
    gen.share_query_across_heads(own)
    q = torch.cat([own.q_lat[0, 0].float(), own.q_pe[0, 0].float()])
    pool = (torch.randn(own.pool.shape[0], 576, generator=torch.Generator().manual_seed(1)) * 8)
    row = q * gap / (float(q @ q) * own.scale * own.kv_scale)
    pool[int(s.prefix[777])] += row
    own.pool = pool.to(torch.float8_e4m3fn).view(torch.uint8).view(own.pool.shape)
    check(join(own, s.prefix), f"gap {gap}")


def test_masked_rows_are_never_read_and_bad_slots_are_reported():
    s = make(1, 16, 500, [40, 9], seed=14)
    for plan in both(s):
        masked_rows(s, plan)


def masked_rows(s, plan):
    want, _ = run(s, plan)
    own = s.own
    nan = own.pool.clone()
    used = torch.cat([s.prefix, own.kv_indices]).long()
    idle = torch.ones(nan.shape[0], dtype=torch.bool)
    idle[used] = False
    nan[idle] = 0x7F   # NaN codes in every row that no table names
    got, _ = run(Shared(dataclasses.replace(own, pool=nan), s.joined, s.prefix), plan)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a bad slot is skipped and reported
    for bad in (-1, own.pool.shape[0], 2 ** 31 - 1, -2 ** 31):
        p = s.prefix.clone()
        p[130] = bad
        (o, lse), ws = run(Shared(own, s.joined, p), plan)
        assert mla.mla_read_device_error(ws) == mla.MLA_DEVERR_BAD_SLOT
        keep = torch.cat([s.prefix[:130], s.prefix[131:]])
        ro, rl = oracle.dense_decode(join(own, keep).joined)
        compare(o, lse, ro, rl, "bad slot")
        idx = own.kv_indices.clone()
        idx[44] = bad   # the fifth of the second request's nine
        (o, lse), ws = run(Shared(dataclasses.replace(own, kv_indices=idx), s.joined, s.prefix),
                           plan)
        assert mla.mla_read_device_error(ws) == mla.MLA_DEVERR_BAD_SLOT
        short = dataclasses.replace(
            own, kv_indices=torch.cat([own.kv_indices[:44], own.kv_indices[45:]]),
            seq_lens=torch.tensor([40, 8]).int(), kv_indptr=torch.tensor([0, 40, 48]).int())
        ro, rl = oracle.dense_decode(join(short, s.prefix).joined)
        compare(o, lse, ro, rl, "bad own slot")


def test_a_query_with_nan_or_inf_stays_in_its_row():
    s = make(1, 16, 400, [30, 5, 60, 2, 9], seed=15)
    want, _ = run(s)
    assert plan_of(s).joined == 1
    q = s.own.q_lat.clone()
    q[1, 3, 7] = float("nan")
    q[2, 0, 500] = float("inf")
    got, _ = run(Shared(dataclasses.replace(s.own, q_lat=q), s.joined, s.prefix))
    same = torch.ones(5, 16, dtype=torch.bool)
    same[1, 3] = same[2, 0] = False
    assert torch.equal(got[0][same.cuda()], want[0][same.cuda()])
    assert torch.equal(got[1][same.cuda()], want[1][same.cuda()])
    for row in ((1, 3), (2, 0)):
        assert bool(torch.isnan(got[0][row]).all()) and bool(torch.isnan(got[1][row]))


@pytest.mark.parametrize("byte", [0x7F, 0xFF])
@pytest.mark.parametrize("column", [0, 300, 511, 570])
def test_a_nan_row_stays_with_the_requests_that_see_it(byte, column):
    # NaN codes in one request's own row, in a tile of four requests
    s = make(1, 16, 400, [30, 5, 260, 2, 9], seed=24)
    assert plan_of(s).joined == 1
    want, _ = run(s)
    pool = s.own.pool.clone()
    slot = int(s.own.kv_indices[35 + 200])   # the third request's
    pool[slot, 0, column] = byte
    got, ws = run(Shared(dataclasses.replace(s.own, pool=pool), s.joined, s.prefix))
    same = torch.arange(5, device="cuda") != 2
    assert torch.equal(got[0][same], want[0][same]) and torch.equal(got[1][same], want[1][same])
    assert bool(torch.isnan(got[0][2]).all()) and bool(torch.isnan(got[1][2]).all())
    assert mla.mla_read_device_error(ws) == 0
    # in the prefix every request sees it, but for the draft rows whose window ends before
    s = make(3, 8, 400, [0, 1, 40], seed=25)
    want, _ = run(s)
    pool = s.own.pool.clone()
    pool[int(s.prefix[398]), 0, column] = byte
    for plan in both(s):
        got, _ = run(Shared(dataclasses.replace(s.own, pool=pool), s.joined, s.prefix), plan)
        blind = torch.zeros(9, dtype=torch.bool, device="cuda")
        blind[0] = True   # request 0, draft 0: positions up to 397
        want, _ = run(s, plan)
        assert torch.equal(got[0][blind], want[0][blind])
        assert bool(torch.isnan(got[0][~blind]).all()) and bool(torch.isnan(got[1][~blind]).all())


def test_repeat_permuted_pool_and_given_outputs():
    s = make(1, 48, 3000, [100, 3, 250, 8], seed=16)
    d, plan = to_cuda(s), plan_of(s)
    ws = mla.workspace(plan)
    (o, lse), _ = run(s, plan, ws, d)
    o2 = torch.empty_like(o)
    (got, none), _ = run(s, plan, ws, d, o=o2, return_lse=False)
    assert got is o2 and none is None and torch.equal(o, o2)
    dirty = torch.full_like(ws, 255)   # whatever the scratch held before
    dirty[:mla.MLA_WORKSPACE_HEADER_BYTES] = 0
    (o3, lse3), _ = run(s, plan, dirty, d)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)
    perm = torch.randperm(s.own.pool.shape[0], generator=torch.Generator().manual_seed(3))
    inv = torch.argsort(perm).int()
    moved = dict(d, pool=s.own.pool[perm].cuda(), prefix_indices=inv[s.prefix.long()].cuda(),
                 kv_indices=inv[s.own.kv_indices.long()].cuda())
    (o4, lse4), _ = run(s, plan, ws, moved)
    assert torch.equal(o, o4) and torch.equal(lse, lse4)


def test_tensors_that_do_not_agree_are_refused():
    """Every wrong tensor here is larger than the right one: it holds what a call would read."""
    s = make(1, 16, 100, [30, 7], seed=91)
    plan, d = plan_of(s), to_cuda(s)
    ws = mla.workspace(plan)
    for name, t in d.items():
        wider = torch.zeros(t.shape, device="cuda",
                            dtype=torch.int64 if t.dtype == torch.int32 else torch.float64)
        longer = torch.cat([t, t])
        apart = torch.stack([t, t], dim=-1)[..., 0]
        for other in (wider, apart) + (() if name == "pool" else (longer,)):
            with pytest.raises(ValueError):
                run(s, plan, ws, dict(d, **{name: other}))
    for kw in (dict(o=torch.empty(4, 16, 512, dtype=torch.bfloat16, device="cuda")),
               dict(o=torch.empty(2, 16, 512, dtype=torch.float32, device="cuda")),
               dict(lse=torch.empty(2, 32, device="cuda")),
               dict(lse=torch.empty(2, 16, dtype=torch.float64, device="cuda"))):
        with pytest.raises(ValueError):
            run(s, plan, ws, d, **kw)


def test_another_stream_and_calls_back_to_back():
    a, b = make(1, 16, 900, [30, 5], seed=17), make(1, 64, 300, [3, 80, 9], seed=18)
    da, db, pa, pb = to_cuda(a), to_cuda(b), plan_of(a), plan_of(b)
    wa, wb = mla.workspace(pa), mla.workspace(pb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(5):   # two streams, a workspace each
        with torch.cuda.stream(side):
            oa = mla.mla_prefix_decode(pa, **da, scale=a.own.scale, kv_scale=a.own.kv_scale,
                                       workspace_t=wa)
        ob = mla.mla_prefix_decode(pb, **db, scale=b.own.scale, kv_scale=b.own.kv_scale,
                                   workspace_t=wb)
        outs.append((oa, ob))
    torch.cuda.synchronize()
    for s, k in ((a, 0), (b, 1)):
        ro, rl = oracle.dense_decode(s.joined)
        for pair in outs:
            compare(*pair[k], ro, rl)
            assert torch.equal(pair[k][0], outs[0][k][0])


def test_pool_past_four_gigabytes():
    rows = 8_000_000
    s = make(1, 16, 300, [20, 4], seed=19)
    own = s.own
    small = own.pool.shape[0]
    spread = (torch.arange(small, dtype=torch.int64) * ((rows - 1) // (small - 1)))
    pool = torch.zeros(rows, 576, dtype=torch.uint8, device="cuda")
    pool[spread.cuda()] = own.pool.view(small, 576).cuda()
    d = to_cuda(s)
    d.update(pool=pool, prefix_indices=spread[s.prefix.long()].int().cuda(),
             kv_indices=spread[own.kv_indices.long()].int().cuda())
    want, _ = run(s)
    got, _ = run(s, d=d)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("seed", range(40))
def test_seeded_random_calls(seed):
    rng = np.random.default_rng(1000 + seed)
    q_len = int(rng.choice([1, 1, 1, 2, 3, 5]))
    heads = int(rng.choice([1, 2, 7, 8, 16, 24, 64, 100, 128]))
    batch = int(rng.integers(1, max(2, min(40, 2000 // (q_len * heads)))))
    P = int(rng.choice([1, 64, 127, 128, 129, 500, 2000, 5000])) + int(rng.integers(0, 130))
    top = int(rng.choice([1, 30, 129, 700]))
    s = make(q_len, heads, P, rng.integers(0, top + 1, batch).tolist(), seed=seed)
    plan = plan_of(s)
    plans = [plan]
    ctas = int(rng.integers(1, 153))
    most = max(1, 152 // plan.tiles)
    for j in (0, 1) if s.own.total_keys else (0,):
        plans.append(variant(plan, ctas=ctas, splits=0, joined=j))
        n = int(rng.integers(1, most + 1))
        plans.append(variant(plan, ctas=plan.tiles * n, splits=n, joined=j))
    ro, rl = oracle.dense_decode(s.joined)
    for p in plans:
        (o, lse), ws = run(s, p)
        compare(o, lse, ro, rl, f"seed {seed} ctas {p.ctas} splits {p.splits} joined {p.joined}")
        assert mla.mla_read_device_error(ws) == 0


def test_a_wait_that_runs_out_ends_the_call():
    s = make(1, 64, 1000, [30, 5], seed=20)
    for plan in both(s) + [variant(plan_of(s), ctas=2, splits=0, joined=1)]:
        wait_runs_out(s, plan)


def wait_runs_out(s, plan):
    ws = mla.workspace(plan)
    mla.mla_debug_wait_limit(300)
    try:
        run(s, plan, ws)
    finally:
        mla.mla_debug_wait_limit(0)
    assert mla.mla_read_device_error(ws) & mla.MLA_DEVERR_TIMEOUT
    mla.mla_workspace_reset(ws)
    check(s, "after a timeout", plan=plan, ws=ws)
