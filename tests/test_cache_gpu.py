"""GPU: the cache operators against plain float64 / integer references.

Tolerances.  A bf16 output is off by at most half a step, 2^-8 of the value; the
fp32 work before that rounding (a chain of at most 72 squares and five shuffle
or elementwise steps, then a few products) stays below 2^-16 of the size of the
terms that a rotation adds, which can be larger than their sum.  An e4m3 value
is off by half a step: 2^-4 of the value, or 2^-10 among the subnormals, after
the same fp32 error.  Copies and tables are exact.
"""
import numpy as np
import pytest
import torch

from split_kv_mla_gb300 import mla

pytestmark = pytest.mark.gpu

SLACK = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _built():
    mla.load()


def e4m3_table():
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def rotate(x, cos, sin, half):
    """(rotated, size of the terms) of x [..., 64] in float64."""
    a, b = (x[..., :32], x[..., 32:]) if half else (x[..., 0::2], x[..., 1::2])
    y, z = a * cos - b * sin, b * cos + a * sin
    m = (a.abs() + b.abs())
    if half:
        return torch.cat([y, z], -1), torch.cat([m, m], -1)
    return torch.stack([y, z], -1).flatten(-2), torch.stack([m, m], -1).flatten(-2)


def normed(x, n, w, eps):
    y = x.clone()
    r = (x[..., :n].square().mean(-1, keepdim=True) + eps).sqrt()
    y[..., :n] = x[..., :n] / r * (1.0 if w is None else w.double())
    return y


def make_append(T, H, width, cols, seed, pool_rows=257, max_pos=1000, slots=None):
    g = torch.Generator().manual_seed(seed)
    bf = torch.bfloat16
    ang = torch.rand(max_pos, 32, generator=g, dtype=torch.float64) * 6.3
    return dict(
        kv=(torch.randn(T, width, generator=g) * 3).to(bf),
        q=torch.randn(T, H, cols, generator=g).to(bf),
        kv_weight=(1 + 0.3 * torch.randn(width, generator=g)).to(bf),
        q_weight=(1 + 0.3 * torch.randn(cols, generator=g)).to(bf),
        positions=torch.randint(0, max_pos, (T,), generator=g).int(),
        cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float(),
        slots=torch.randperm(pool_rows, generator=g)[:T].int() if slots is None else slots,
        pool=torch.randint(0, 127, (pool_rows, width), generator=g).to(torch.uint8))


def reference_append(c, norm_cols, q_norm, half, kv_scale, eps, weights=True):
    """Float64 values before rounding and the size of their terms."""
    W, D = c["kv"].shape[1], c["q"].shape[2]
    cs = c["cos_sin"].double()[c["positions"].long()]
    cos, sin = cs[:, :32], cs[:, 32:]
    kv = c["kv"].double()
    if norm_cols:
        kv = normed(kv, norm_cols, c["kv_weight"][:norm_cols] if weights else None, eps)
    size = kv.abs()
    kv[:, W - 64:], size[:, W - 64:] = rotate(kv[:, W - 64:], cos, sin, half)
    q = c["q"].double()
    if q_norm:
        q = normed(q, D, c["q_weight"] if weights else None, eps)
    qsize = q.abs()
    q[..., D - 64:], qsize[..., D - 64:] = rotate(q[..., D - 64:], cos[:, None], sin[:, None], half)
    return kv / kv_scale, size / abs(kv_scale), q, qsize


def check_bf16(got, want, size):
    err = (got.cpu().double() - want).abs()
    assert bool((err <= want.abs() * 2.0 ** -8 + size * SLACK).all()), err.max()


def check_e4m3(got_bytes, want, size):
    got = e4m3_table()[got_bytes.cpu().int()]
    want = want.clamp(-448, 448)
    half = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10).double())
    err = (got - want).abs()
    assert bool((err <= half + size * SLACK).all()), (err - half).max()


def run_append(c, norm_cols, q_norm, half, kv_scale, eps=1e-6, weights=True, **kw):
    d = {k: v.cuda() for k, v in c.items()}
    ws = mla.cache_workspace()
    nope, pe = mla.mla_cache_append(
        d["kv"], d["slots"], d["pool"], d["positions"], d["cos_sin"], kv_scale, q=d["q"],
        kv_weight=d["kv_weight"][:norm_cols] if norm_cols and weights else None,
        kv_norm_cols=norm_cols, q_weight=d["q_weight"] if q_norm and weights else None,
        q_norm=q_norm, eps=eps, half_split=half, workspace_t=ws, **kw)
    torch.cuda.synchronize()
    return nope, pe, d["pool"], mla.mla_read_device_error(ws)


def check_append(c, out, norm_cols, q_norm, half, kv_scale, eps=1e-6, weights=True):
    nope, pe, pool, _ = out
    kv, size, q, qsize = reference_append(c, norm_cols, q_norm, half, kv_scale, eps, weights)
    D = q.shape[2]
    check_bf16(pe, q[..., D - 64:], qsize[..., D - 64:])
    if D > 64:
        check_bf16(nope, q[..., :D - 64], qsize[..., :D - 64])
    else:
        assert nope is None
    on = c["slots"] >= 0
    check_e4m3(pool[c["slots"][on].long().cuda()], kv[on], size[on])
    rest = torch.ones(c["pool"].shape[0], dtype=torch.bool)
    rest[c["slots"][on].long()] = False
    assert torch.equal(pool.cpu()[rest], c["pool"][rest])


@pytest.mark.parametrize("T,H,width,cols,norm,q_norm,half", [
    (1, 1, 576, 64, 512, False, False), (1, 16, 576, 192, 512, True, True),
    (7, 3, 576, 64, 0, True, False), (33, 5, 576, 128, 576, True, False),
    (31, 128, 576, 64, 512, False, True), (64, 16, 576, 192, 512, False, False),
    (5, 9, 576, 256, 512, True, True), (3, 2, 576, 320, 512, True, False),
    (3, 2, 576, 384, 0, False, True), (3, 7, 576, 448, 512, True, False),
    (129, 4, 576, 576, 576, True, True), (1, 64, 512, 512, 512, True, False),
    (45, 17, 512, 512, 448, True, True), (200, 1, 512, 512, 0, False, False),
    (17, 6, 512, 64, 512, False, False)])
def test_append(T, H, width, cols, norm, q_norm, half):
    c = make_append(T, H, width, cols, seed=T * 131 + H)
    out = run_append(c, norm, q_norm, half, 0.03125)
    assert out[3] == 0
    check_append(c, out, norm, q_norm, half, 0.03125)


@pytest.mark.parametrize("kv_scale", [1.0, 0.0173, -0.5])
def test_append_without_weights_and_scales(kv_scale):
    c = make_append(20, 4, 576, 192, seed=5)
    out = run_append(c, 512, True, False, kv_scale, weights=False)
    check_append(c, out, 512, True, False, kv_scale, weights=False)


def test_append_rows_or_queries_alone_and_padding():
    c = make_append(40, 8, 576, 192, seed=6)
    c["slots"][::3] = -1
    out = run_append(c, 512, True, False, 0.25)
    check_append(c, out, 512, True, False, 0.25)
    d = {k: v.cuda() for k, v in c.items()}
    pool = d["pool"].clone()
    got = mla.mla_cache_append(d["kv"], d["slots"], pool, d["positions"], d["cos_sin"], 0.25,
                               kv_weight=d["kv_weight"][:512], kv_norm_cols=512)
    assert got == (None, None) and torch.equal(pool, out[2])
    nope, pe = mla.mla_cache_append(None, None, None, d["positions"], d["cos_sin"], q=d["q"],
                                    q_weight=d["q_weight"], q_norm=True)
    assert torch.equal(nope, out[0]) and torch.equal(pe, out[1])
    nothing = mla.mla_cache_append(d["kv"][:0], d["slots"][:0], pool, d["positions"][:0],
                                   d["cos_sin"], q=d["q"][:0])
    assert nothing[1].shape == (0, 8, 64)


def test_append_strided_inputs_and_given_outputs():
    # kv and q as slices of wider projections, heads outermost, a [N, 1, W] fp8 cache
    T, H = 19, 6
    c = make_append(T, H, 576, 192, seed=7)
    want = run_append(c, 512, True, True, 0.125)
    d = {k: v.cuda() for k, v in c.items()}
    wide = torch.full((T, 1536 + 576), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 1536:] = d["kv"]
    qt = torch.empty(H, T, 200, dtype=torch.bfloat16, device="cuda").fill_(9.0)
    qt[..., :192] = d["q"].transpose(0, 1)
    pool = d["pool"].view(257, 1, 576).view(torch.float8_e4m3fn)
    nope = torch.empty(T * H, 128, dtype=torch.bfloat16, device="cuda")
    pe = torch.empty(T, H, 64, dtype=torch.bfloat16, device="cuda")
    got = mla.mla_cache_append(wide[:, 1536:], d["slots"], pool, d["positions"], d["cos_sin"],
                               0.125, q=qt.transpose(0, 1)[..., :192],
                               kv_weight=d["kv_weight"][:512], kv_norm_cols=512,
                               q_weight=d["q_weight"], q_norm=True, half_split=True,
                               q_nope=nope, q_pe=pe)
    assert got[0] is nope and got[1] is pe
    assert torch.equal(nope.view(T, H, 128), want[0]) and torch.equal(pe, want[1])
    assert torch.equal(pool.view(torch.uint8).view(257, 576), want[2])
    with pytest.raises(ValueError):
        mla.mla_cache_append(d["kv"].t().contiguous().t(), d["slots"], d["pool"], d["positions"],
                             d["cos_sin"])
    with pytest.raises(mla.MlaError):   # rows 20 bytes apart from a 16-byte step
        odd = torch.zeros(T, 577, dtype=torch.bfloat16, device="cuda")[:, :576]
        mla.mla_cache_append(odd, d["slots"], d["pool"], d["positions"], d["cos_sin"])


def test_append_reports_bad_slots_and_positions():
    c = make_append(24, 4, 576, 64, seed=8)
    c["slots"][3] = 257
    c["slots"][4] = 2 ** 31 - 1
    out = run_append(c, 512, False, False, 0.25)
    assert out[3] == mla.MLA_DEVERR_BAD_SLOT
    good = dict(c, slots=c["slots"].clone())
    good["slots"][3:5] = -1
    check_append(good, out, 512, False, False, 0.25)
    for bad in (1000, -1, -2 ** 31, 2 ** 31 - 1):
        p = good["positions"].clone()
        p[7] = bad
        pe = torch.full((24, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        got = run_append(dict(good, positions=p), 512, False, False, 0.25, q_pe=pe)
        assert got[3] == mla.MLA_DEVERR_BAD_POSITION
        assert bool((pe[7] == 5).all())
        same = torch.arange(24) != 7
        assert torch.equal(pe[same.cuda()], out[1][same.cuda()])
        slot = int(good["slots"][7])
        if slot >= 0:
            assert torch.equal(got[2][slot].cpu(), c["pool"][slot])


def test_append_extremes_stay_in_their_row():
    c = make_append(12, 3, 576, 192, seed=9)
    clean = run_append(c, 512, True, False, 0.03125)
    kv, q = c["kv"].clone(), c["q"].clone()
    kv[2] = 0                       # a zero row is 0 / sqrt(eps)
    kv[4, 100] = float("inf")       # inf / inf
    kv[5, 570] = float("nan")       # in the RoPE part, past the norm
    kv[6] = 3e30                    # saturates where it is not normed
    q[7, 1, 5] = float("nan")
    got = run_append(dict(c, kv=kv, q=q), 512, True, False, 0.03125)
    rows = {t: int(c["slots"][t]) for t in range(12)}
    for t in (0, 1, 3, 7, 8, 9, 10, 11):
        assert torch.equal(got[2][rows[t]], clean[2][rows[t]])
    vals = e4m3_table()
    r2 = vals[got[2][rows[2]].cpu().int()]
    assert bool((r2 == 0).all())
    r4 = vals[got[2][rows[4]].cpu().int()]
    assert bool(torch.isnan(r4[100])) and bool((r4[:100] == 0).all())
    r5 = vals[got[2][rows[5]].cpu().int()]
    assert int(torch.isnan(r5).sum()) == 2 and bool(torch.isnan(r5[570:572]).all())
    r6 = vals[got[2][rows[6]].cpu().int()]
    assert bool((r6[512:].abs() == 448).all()) and not bool(torch.isnan(r6).any())
    other = torch.ones(12, 3, dtype=torch.bool)
    other[7, 1] = False
    assert torch.equal(got[1][other.cuda()], clean[1][other.cuda()])
    assert bool(torch.isnan(got[1][7, 1]).all())


def test_append_past_two_gigabytes():
    # rows beyond 2^31 bytes of the pool and of the queries' table
    rows = 4_000_000
    c = make_append(6, 2, 576, 64, seed=10)
    c["slots"] = torch.tensor([rows - 1, 3_800_000, 0, 3_728_270, 3_728_271, 5]).int()
    pool = torch.zeros(rows, 576, dtype=torch.uint8, device="cuda")
    d = {k: v.cuda() for k, v in c.items() if k != "pool"}
    mla.mla_cache_append(d["kv"], d["slots"], pool, d["positions"], d["cos_sin"], 0.25, q=d["q"],
                         kv_weight=d["kv_weight"][:512], kv_norm_cols=512)
    kv, size, _, _ = reference_append(c, 512, False, False, 0.25, 1e-6)
    check_e4m3(pool[d["slots"].long()], kv, size)
    assert int((pool != 0).any(1).sum()) == 6


def test_append_in_a_graph_and_on_another_stream():
    c = make_append(16, 4, 576, 192, seed=11)
    d = {k: v.cuda() for k, v in c.items()}
    ws = mla.cache_workspace()

    def call():
        return mla.mla_cache_append(d["kv"], d["slots"], d["pool"], d["positions"], d["cos_sin"],
                                    0.25, q=d["q"], kv_weight=d["kv_weight"][:512],
                                    kv_norm_cols=512, workspace_t=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    check_append(c, (*call(), d["pool"], 0), 512, False, False, 0.25)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nope, pe = call()
    new = make_append(16, 4, 576, 192, seed=12)
    for k in ("kv", "q", "positions"):
        d[k].copy_(new[k])
    graph.replay()
    torch.cuda.synchronize()
    want = dict(c, kv=new["kv"], q=new["q"], positions=new["positions"])
    check_append(want, (nope, pe, d["pool"], 0), 512, False, False, 0.25)


# ---- fork -----------------------------------------------------------------------------------

def make_fork(lens, parents, keep, n, pool_rows, width, seed):
    """Parents of `lens` positions; child f takes n[f] of parents[f]."""
    g = torch.Generator().manual_seed(seed)
    fresh_n = [max(0, n[f] - max(0, keep[f])) for f in range(len(parents))]
    perm = torch.randperm(pool_rows, generator=g).int()
    total = sum(lens)
    ptr = lambda x: torch.tensor([0] + list(np.cumsum(x)) if len(x) else [0]).int()  # noqa: E731
    return dict(pool=torch.randint(0, 256, (pool_rows, width), generator=g).to(torch.uint8),
                kv_indices=perm[:total].clone(), kv_indptr=ptr(lens),
                parents=torch.tensor(parents).int(), keep=torch.tensor(keep).int(),
                child_indptr=ptr(n), fresh=perm[total:total + sum(fresh_n)].clone(),
                fresh_indptr=ptr(fresh_n))


def reference_fork(c):
    pool = c["pool"].clone()
    table = []
    for f in range(c["parents"].numel()):
        p = int(c["parents"][f])
        base = int(c["kv_indptr"][p])
        for j in range(int(c["child_indptr"][f + 1] - c["child_indptr"][f])):
            src = int(c["kv_indices"][base + j])
            k = max(0, int(c["keep"][f]))
            if j < k:
                table.append(src)
            else:
                dst = int(c["fresh"][int(c["fresh_indptr"][f]) + j - k])
                pool[dst] = c["pool"][src]
                table.append(dst)
    return torch.tensor(table).int(), pool


def run_fork(c, **kw):
    d = {k: v.cuda() for k, v in c.items()}
    ws = mla.cache_workspace()
    table = mla.mla_cache_fork(d["pool"], d["kv_indices"], d["kv_indptr"], d["parents"],
                               d["keep"], d["child_indptr"], int(c["child_indptr"][-1]),
                               d["fresh"], d["fresh_indptr"], workspace_t=ws, **kw)
    torch.cuda.synchronize()
    return table, d["pool"], mla.mla_read_device_error(ws)


@pytest.mark.parametrize("lens,parents,keep,n,width", [
    ([1], [0], [0], [1], 576), ([1], [0], [1], [1], 512),
    ([5, 0, 9], [2, 0, 2], [4, 0, 9], [9, 5, 9], 576),
    ([100], [0] * 9, list(range(0, 90, 10)), [100] * 9, 512),
    ([40, 77, 3], [1, 1, 0, 2, 0], [70, -3, 100, 2, 0], [77, 30, 39, 3, 0], 576),
    ([0, 0], [0, 1], [0, 3], [0, 0], 576),
    ([2049, 700], [0, 1, 0, 1, 0, 0, 1], [2048, 1, 1000, 699, 2049, 0, 350],
     [2049, 700, 1500, 700, 2049, 2049, 351], 576)])
def test_fork(lens, parents, keep, n, width):
    c = make_fork(lens, parents, keep, n, sum(lens) + sum(n) + 13, width, seed=len(n) + sum(n))
    table, pool, err = run_fork(c)
    want_table, want_pool = reference_fork(c)
    assert err == 0
    assert torch.equal(table.cpu(), want_table)
    assert torch.equal(pool.cpu(), want_pool)


def test_fork_of_many_entries():
    # above 131072 entries a warp takes 32 of them, below 8
    lens, F = [3001, 2999, 1], 60
    parents = [f % 3 for f in range(F)]
    n = [lens[p] for p in parents]
    keep = [(f * 977) % 3100 for f in range(F)]
    c = make_fork(lens, parents, keep, n, 130000, 512, seed=1)
    small = make_fork(lens, parents[:40], keep[:40], n[:40], 130000, 576, seed=2)
    assert sum(n[:40]) < 1 << 17 and sum(n) < 1 << 17
    big = make_fork([30011], [0] * 5, [30000, 1, 15000, 29999, 12345], [30011] * 5, 130000, 576, 3)
    assert int(big["child_indptr"][-1]) > 1 << 17
    for case in (c, small, big):
        table, pool, err = run_fork(case)
        want_table, want_pool = reference_fork(case)
        assert err == 0
        assert torch.equal(table.cpu(), want_table)
        assert torch.equal(pool.cpu(), want_pool)


def test_fork_reports_and_skips_what_is_out_of_range():
    c = make_fork([50, 60], [0, 1, 0], [10, 60, 50], [50, 60, 50], 300, 576, seed=3)
    _, want_pool = reference_fork(c)
    bad = {k: v.clone() for k, v in c.items()}
    bad["parents"][1] = 2
    table, pool, err = run_fork(bad)
    assert err == mla.MLA_DEVERR_BAD_TABLE
    assert bool((table[50:110] == -1).all()) and torch.equal(pool.cpu(), want_pool)
    bad = {k: v.clone() for k, v in c.items()}
    bad["child_indptr"][3] = 165   # five positions past the parent's 50
    table, pool, err = run_fork(bad)
    assert err == mla.MLA_DEVERR_BAD_LENGTH
    assert bool((table[160:] == -1).all()) and torch.equal(pool.cpu(), want_pool)
    bad = {k: v.clone() for k, v in c.items()}
    bad["fresh"][4] = 300
    bad["kv_indices"][20] = -7
    table, pool, err = run_fork(bad)
    assert err == mla.MLA_DEVERR_BAD_SLOT
    skip = torch.tensor([int(c["fresh"][4]), int(c["fresh"][10])])
    want = want_pool.clone()
    want[skip] = c["pool"][skip]
    assert torch.equal(pool.cpu(), want)
    assert int(table[14]) == 300 and int(table[20]) == int(c["fresh"][10])
    bad = {k: v.clone() for k, v in c.items()}
    bad["fresh_indptr"][1:] = 39   # one fresh slot short
    table, pool, err = run_fork(bad)
    assert err == mla.MLA_DEVERR_BAD_TABLE and int(table[49]) == -1
    # entries of a given table past the last child's are left alone
    given = torch.full((200,), 77, dtype=torch.int32, device="cuda")
    table, pool, err = run_fork(c, table=given)
    assert err == 0 and bool((table[160:] == 77).all())


def test_fork_past_four_gigabytes():
    rows = 8_000_000
    pool = torch.zeros(rows, 576, dtype=torch.uint8, device="cuda")
    src = torch.tensor([0, 7_900_000, 11]).int()
    vals = torch.randint(1, 255, (3, 576), dtype=torch.uint8)
    pool[src.long().cuda()] = vals.cuda()
    dst = torch.tensor([rows - 1, 12, 7_456_541]).int()
    i = lambda *x: torch.tensor(x).int().cuda()  # noqa: E731
    table = mla.mla_cache_fork(pool, src.cuda(), i(0, 3), i(0), i(0), i(0, 3), 3, dst.cuda(),
                               i(0, 3))
    assert torch.equal(table.cpu(), dst)
    assert torch.equal(pool[dst.long().cuda()].cpu(), vals)
    assert int((pool[::1000] != 0).any(1).sum()) == int((torch.cat([src, dst]) % 1000 == 0).sum())


# ---- compaction -------------------------------------------------------------------------------

def reference_compact(pool, idx):
    n = pool.shape[0]
    live = sorted({int(s) for s in idx if 0 <= s < n})
    count = len(live)
    named = set(live)
    holes = [s for s in range(count) if s not in named]
    to = dict(zip([s for s in live if s >= count], holes))
    out = pool.clone()
    for s, d in to.items():
        out[d] = pool[s]
    table = [to.get(int(s), int(s)) for s in idx]
    return out, torch.tensor(table).int(), count


def check_compact(pool, idx, in_place=False):
    want_pool, want_table, want = reference_compact(pool, idx)
    d_pool, d_idx = pool.cuda(), idx.cuda()
    ws = mla.cache_workspace(pool.shape[0])
    for again in range(2):   # a second call on the result moves nothing
        out = d_idx if in_place else None
        table, live = mla.mla_cache_compact(d_pool, d_idx, new_indices=out, workspace_t=ws)
        torch.cuda.synchronize()
        assert torch.equal(table.cpu(), want_table)
        assert int(live) == want
        assert torch.equal(d_pool.cpu(), want_pool)
        d_idx = table
    return mla.mla_read_device_error(ws)


@pytest.mark.parametrize("rows,live,width", [
    (1, 1, 576), (1, 0, 576), (2, 1, 512), (31, 16, 576), (32, 32, 576), (33, 1, 512),
    (64, 40, 576), (1000, 0, 576), (1000, 1000, 576), (8192, 4096, 512), (8193, 1, 576),
    (8193, 8192, 576), (20000, 3000, 576), (20000, 17000, 576), (70001, 35000, 512)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(rows, live, width, in_place):
    g = torch.Generator().manual_seed(rows + live)
    pool = torch.randint(0, 256, (rows, width), generator=g).to(torch.uint8)
    slots = torch.randperm(rows, generator=g)[:live].int()
    idx = torch.cat([slots, slots[:live // 3], torch.tensor([-1, -5]).int()])
    assert check_compact(pool, idx, in_place) == 0


@pytest.mark.parametrize("place", ["tail", "head", "middle", "borders"])
def test_compact_where_the_live_rows_lie(place):
    n = 3 * 8192 + 17
    g = torch.Generator().manual_seed(4)
    pool = torch.randint(0, 256, (n, 576), generator=g).to(torch.uint8)
    idx = {"tail": torch.arange(n - 9000, n), "head": torch.arange(9000),
           "middle": torch.arange(8000, 17000),
           "borders": torch.tensor([0, 31, 32, 8191, 8192, 16383, 16384, n - 1])}[place]
    assert check_compact(pool, idx.int().flip(0)) == 0


@pytest.mark.parametrize("rows,entries", [(16384, 32768), (16385, 9000), (16384, 32769),
                                          (500, 40000), (262144, 100000), (262145, 120000),
                                          (300000, 120000), (1048576, 500000), (1048577, 300001),
                                          (1300000, 700001), (100000, 0)])
def test_compact_both_sides_of_the_small_pool_rule(rows, entries):
    # up to 16384 rows and 32768 entries one CTA ranks the pool, above kernels do, with
    # counts of chunks above 262144 rows
    g = torch.Generator().manual_seed(rows)
    pool = torch.randint(0, 256, (rows, 512), generator=g).to(torch.uint8)
    slots = torch.randint(0, rows, (entries,), generator=g).int()
    assert check_compact(pool, slots) == 0


def test_compact_one_entry_many_times_and_out_of_range():
    pool = torch.randint(0, 256, (500, 576), dtype=torch.uint8)
    assert check_compact(pool, torch.full((3000,), 499).int()) == 0
    idx = torch.tensor([499, 500, 3, -2, 2 ** 31 - 1, 499]).int()
    assert check_compact(pool, idx) == mla.MLA_DEVERR_BAD_SLOT
    assert check_compact(pool, torch.empty(0).int()) == 0


def test_compact_past_four_gigabytes_and_in_a_graph():
    rows = 8_000_000
    pool = torch.zeros(rows, 576, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([rows - 1, 7_999_000, 2, 7_456_541, 4]).int().cuda()
    vals = torch.randint(1, 255, (5, 576), dtype=torch.uint8).cuda()
    pool[slots.long()] = vals
    ws = mla.cache_workspace(rows)
    keep = pool[rows - 2000:].clone()

    def call():
        return mla.mla_cache_compact(pool, slots, workspace_t=ws)
    table, live = call()
    assert int(live) == 5
    assert table.tolist() == [3, 1, 2, 0, 4]   # tail rows in slot order into holes 0, 1, 3
    assert torch.equal(pool[table.long()], vals)
    assert torch.equal(pool[rows - 2000:], keep)   # rows past L keep their bytes
    pool[:2] = 0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        table, live = call()
    for _ in range(2):
        pool[:2] = 0
        graph.replay()
        assert table.tolist() == [3, 1, 2, 0, 4] and int(live) == 5
        assert torch.equal(pool[table.long()], vals)
    slots[0] = 5   # other entries, the same graph
    graph.replay()
    # row 5 is a tail row now, the first
    assert table.tolist() == [0, 3, 2, 1, 4] and int(live) == 5
    assert torch.equal(pool[table.long()][1:], vals[1:])
    assert mla.mla_read_device_error(ws) == 0
