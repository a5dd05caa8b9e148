"""GPU: beam selection against float64.

A score is cum + x - ln sum e^x, rounded to fp32: half a step, 2^-24 of its value.  The
sum behind it is fp32: with d the distance of a term's logit from its segment's maximum,
a term e^-d carries 2 d 2^-24 from the rounding of d and of its product with log2 e, and
2^-22 from the exponential; the mean of d over the terms is at most ln(2048) plus what
the maximum's own term does not have, below 20 for these inputs; at most 40 additions in
a row (32 of a lane's logits, 5 of the lanes) and 40 for a row's segments follow.  That
is at most (40 + 4 + 80) 2^-24 < 2^-17 of the sum, and of ln of it; ln itself and the
sum of the parts add less than 2^-22.  So a score is off by at most 2^-24 |score| + 2^-16.
Where candidates lie further apart than twice that, their order is the exact one; ties
that the inputs make exact go to the lower index.
"""
import math

import pytest
import torch

from split_kv_mla_gb300 import mla

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    mla.load()


def slack(score):
    return score.abs() * 2.0 ** -24 + 2.0 ** -16


def exact_scores(logits, scores, finished=None, end=-1):
    """float64 [B, W * V]; -inf where there is no candidate."""
    B, W = scores.shape
    x = logits.cpu().double()
    cum = scores.cpu().double().view(-1, 1)
    d = x - x.amax(-1, keepdim=True)
    s = cum + (d - torch.log(torch.exp(d).sum(-1, keepdim=True)))
    bad = ~(x < math.inf).all(-1, keepdim=True) | ~(cum < math.inf)
    s = torch.where(bad | (cum == -math.inf) | (x == -math.inf), -math.inf, s)
    if finished is not None:
        for r in finished.cpu().view(-1).bool().nonzero()[:, 0].tolist():
            s[r] = -math.inf
            s[r, end] = cum[r, 0]
    return s.view(B, -1)


def run(logits, scores, K=None, ws=None, **kw):
    B, W = scores.shape
    ws = mla.beam_workspace(B, W, logits.shape[1]) if ws is None else ws
    out = mla.mla_beam_select(logits, scores, K, workspace_t=ws, **kw)
    torch.cuda.synchronize()
    return out, mla.mla_read_device_error(ws)


def check(out, want, W, V, finished=None, end=-1):
    tokens, parents, scores = (t.cpu() for t in out[:3])
    B, K = tokens.shape
    for b in range(B):
        n = min(K, int((want[b] > -math.inf).sum()))
        at = (parents[b].long() - b * W) * V + tokens[b].long()
        assert bool((tokens[b, n:] == -1).all()) and bool((parents[b, n:] == b * W).all())
        assert bool((scores[b, n:] == -math.inf).all())
        at = at[:n]
        assert at.unique().numel() == n
        got, ref = scores[b, :n].double(), want[b][at]
        assert bool(((got - ref).abs() <= slack(ref)).all()), (got - ref).abs().max()
        # in order, equal scores by index
        step = scores[b, 1:n] - scores[b, :n - 1]
        assert bool((step <= 0).all()) and bool(((step < 0) | (at[1:] > at[:-1])).all())
        # the best there are: nothing outside beats the last by more than both are off
        top = torch.topk(want[b], n)
        if n:
            assert bool(((top.values - got).abs() <= slack(top.values)).all())
        apart = torch.full((n,), True)
        more = torch.topk(want[b], min(want[b].numel(), n + 1)).values
        gap = more[:-1] - more[1:] > 4 * slack(more[:-1])
        apart[:gap.numel()] &= gap[:n]
        apart[1:] &= gap[:n - 1] if n else gap[:0]
        assert torch.equal(at[apart], top.indices[apart])
        if out[3] is not None:
            ends = torch.ones(K, dtype=torch.bool)
            ends[:n] = tokens[b, :n] == end
            if finished is not None:
                ends[:n] |= finished.cpu().view(-1).bool()[parents[b, :n].long()]
            assert torch.equal(out[3][b].cpu().bool(), ends)


def make(B, W, V, dtype, seed, pad=0, offset=0, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    flat = torch.empty(B * W * (V + pad) + offset, dtype=dtype)
    x = flat[offset:].view(B * W, V + pad)
    x.copy_(torch.randn(B * W, V + pad, generator=g) * spread)
    flat = flat.cuda()
    return flat[offset:].view(B * W, V + pad)[:, :V], (-30 * torch.rand(B, W, generator=g)).cuda()


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("B,W,V,K,pad,offset", [
    (1, 1, 1, 1, 0, 0), (1, 1, 2, 4, 0, 0), (3, 2, 7, 5, 0, 0), (2, 3, 8, 3, 0, 0),
    (2, 3, 9, 32, 0, 0), (1, 4, 255, 4, 0, 0), (1, 4, 256, 4, 0, 0), (1, 4, 257, 8, 0, 0),
    (2, 5, 1023, 5, 0, 0), (2, 5, 1024, 10, 0, 0), (2, 5, 1025, 10, 0, 0), (1, 32, 2047, 32, 0, 0),
    (1, 8, 2048, 8, 8, 0), (3, 8, 2049, 16, 0, 0), (2, 8, 5003, 16, 0, 3), (1, 4, 32000, 4, 0, 0),
    (2, 8, 50001, 16, 0, 0), (1, 2, 200003, 32, 5, 7), (5, 1, 4096, 1, 0, 1), (2, 2, 4100, 3, 4, 4),
    (300, 3, 700, 3, 0, 0), (1, 2, 1 << 20, 4, 0, 0),
    # beams far apart of a small vocabulary: one or two of them hold all of the best
    (37, 16, 1084, 16, 0, 0), (13, 8, 1532, 8, 76, 0), (2, 8, 1247, 16, 0, 1), (7, 5, 1822, 10, 0, 0),
    # more groups and parts than a thread keeps
    (1, 16, 300001, 32, 0, 0), (1, 32, 140000, 32, 0, 0), (2, 1, 1000003, 5, 0, 1)])
def test_random(dtype, B, W, V, K, pad, offset):
    x, s = make(B, W, V, dtype, seed=B + 7 * W + 11 * V, pad=pad, offset=offset)
    out, err = run(x, s, K)
    assert err == 0 and out[3] is None
    check(out, exact_scores(x, s), W, V)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shift", range(8))
def test_every_alignment(dtype, shift):
    for V in (2048, 4099, 2561):
        x, s = make(2, 3, V, dtype, seed=shift, offset=shift)
        out, err = run(x, s, 6)
        assert err == 0
        check(out, exact_scores(x, s), 3, V)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("V", [300, 4099, 65536])
def test_masks(dtype, V):
    W, K = 6, 12
    x, s = make(2, W, V, dtype, seed=V)
    x[0] = -math.inf                     # nothing is left of this row
    x[1, 1:] = -math.inf                 # one token
    x[2, : V // 2] = -math.inf
    x[3, V // 3:] = -math.inf
    x[4, ::2] = -math.inf
    x[5, torch.rand(V, device="cuda") < 0.999] = -math.inf
    x[W:2 * W] = -math.inf               # the second request has three candidates
    x[W + 2, V - 1] = 1.0
    x[W + 2, 17] = 1.0
    x[W + 4, 0] = -7.0
    out, err = run(x, s, K, end_token=17)
    assert err == 0
    check(out, exact_scores(x, s), W, V, end=17)
    assert int((out[0][1] >= 0).sum()) == 3
    low = torch.finfo(dtype).min         # masked by the type's lowest value: still candidates
    y, s = make(1, 2, 300, dtype, seed=1)
    y[0] = low
    y[1, 5:] = low
    out, err = run(y, s, 20)
    assert err == 0
    check(out, exact_scores(y, s), 2, 300)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_finished_and_unused_beams(dtype):
    B, W, V, end = 4, 4, 3001, 2
    x, s = make(B, W, V, dtype, seed=9)
    s -= 10
    done = torch.zeros(B, W, dtype=torch.bool, device="cuda")
    done[0, 1] = done[1, 0] = done[1, 3] = True
    done[2] = True                       # all of them
    s[0, 1], s[3, 1:] = -0.5, -math.inf  # the best; a first step
    s[1, 3] = -math.inf                  # finished, and no beam
    x[1] = math.nan                      # of beams whose logits are not looked at
    x[7] = math.inf
    x[13:] = math.nan
    for kind in (torch.bool, torch.uint8):
        out, err = run(x, s, 6, finished=done.to(kind), end_token=end)
        assert err == 0
        want = exact_scores(torch.nan_to_num(x.float(), posinf=1.0), s, done, end)
        check(out, want, W, V, done, end)
    assert out[0][0, 0] == end and out[1][0, 0] == 1 and out[2][0, 0] == -0.5
    assert bool((out[2][2, :4] == s[2].sort(descending=True).values).all())
    assert out[0][2].tolist() == [end] * 4 + [-1] * 2 and bool(out[3][2].all())


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("bad", ["nan", "inf", "all nan", "all inf", "score nan", "score inf"])
def test_bad_numbers_stay_in_their_beam(dtype, bad):
    W, V = 3, 5001
    x, s = make(2, W, V, dtype, seed=4)
    if bad.startswith("score"):
        s[0, 1] = float(bad.split()[1])
    elif bad.startswith("all"):
        x[1] = float(bad.split()[1])
    else:
        x[1, 4321] = float(bad)
    out, err = run(x, s, 3)
    assert err == mla.MLA_DEVERR_BAD_LOGITS
    keep = torch.tensor([0, 2, 3, 4, 5])
    want = exact_scores(x, s).view(6, V)
    clean = exact_scores(torch.nan_to_num(x.float(), nan=0.0, posinf=0.0),
                         torch.nan_to_num(s, nan=0.0, posinf=0.0)).view(6, V)
    assert bool((want[1] == -math.inf).all()) and torch.equal(want[keep], clean[keep])
    check(out, want.view(2, W * V), W, V)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("V", [5, 256, 4099, 100001])
def test_ties_go_to_the_lower_index(dtype, V):
    K = 7
    x = torch.zeros(2 * 3, V, dtype=dtype, device="cuda")
    s = torch.full((2, 3), -4.0, device="cuda")
    s[1, 0] = -5.0
    out, err = run(x, s, K)
    assert err == 0
    first = [(w, v) for w in range(3) for v in range(V)][:K]
    assert out[0][0].tolist() == [v for _, v in first]
    assert out[1][0].tolist() == [w for w, _ in first]
    second = [(w, v) for w in (1, 2) for v in range(V)][:K]
    assert out[0][1].tolist() == [v for _, v in second]
    assert out[1][1].tolist() == [3 + w for w, _ in second]
    assert bool((out[2][0] == out[2][0, 0]).all())
    # equal beams, each at an alignment of its own: the first one's candidate is first
    g = torch.Generator().manual_seed(V)
    row = (torch.randn(V, generator=g) * 3).to(dtype).cuda()
    flat = torch.empty(8 * (V + 1) + 3, dtype=dtype, device="cuda")
    y = flat[3:].view(8, V + 1)[:, :V]
    y.copy_(row.expand(8, V))
    out, err = run(y, torch.full((1, 8), -1.25, device="cuda"), 16)
    order = torch.sort(row.float(), descending=True, stable=True)
    want = []
    for value in order.values.unique().flip(0).tolist():
        tied = order.indices[order.values == value].tolist()
        want += [(w, v) for w in range(8) for v in tied]
        if len(want) >= 16:
            break
    # (a value's tokens beam by beam: the lower w * V + v)
    assert list(zip(out[1][0].tolist(), out[0][0].tolist())) == want[:16][:out[0].numel()]


@pytest.mark.parametrize("dtype", [BF, FP])
def test_many_candidates_in_few_groups(dtype):
    # the best of 32 groups is low, and eight groups of 256 lie above it
    V = 64 * 256
    x, s = make(1, 1, V, dtype, seed=2)
    x -= 40
    x[0, 2048:4096] += 50
    out, err = run(x, s, 32)
    assert err == 0
    check(out, exact_scores(x, s), 1, V)
    # a descending row: the first group has all of the best
    x[0] = torch.linspace(9, -9, V, device="cuda").to(dtype)
    out, err = run(x, s, 32)
    check(out, exact_scores(x, s), 1, V)
    # two thousand groups, and none in the columns of some warp's share
    x, s = make(1, 8, 65536, dtype, seed=3)
    x[3, 224 * 256:] = -math.inf
    x[7, 224 * 256:] = -math.inf
    out, err = run(x, s, 32)
    assert err == 0
    check(out, exact_scores(x, s), 8, 65536)


def test_large_values_and_scores():
    x, s = make(2, 4, 3000, FP, seed=6)
    x[0] *= 1e30
    x[1] = 3e38
    x[2] = -3e38
    x[3] += 1e6
    x[4] *= 100.0
    s[1] = torch.tensor([-1e30, 0.0, 1e4, -1e-30])
    out, err = run(x, s, 8)
    assert err == 0
    check(out, exact_scores(x, s), 4, 3000)


def test_logits_behind_four_gigabytes():
    # rows 2^28 elements apart: the last starts at 2^32 bytes and more
    stride, V, W = 1 << 28, 5001, 16
    buf = torch.empty(stride * (W - 1) + V, dtype=BF, device="cuda")
    x = buf.as_strided((W, V), (stride, 1))
    y, s = make(1, W, V, BF, seed=12)
    x.copy_(y)
    s[0] = torch.linspace(-9, 0, W, device="cuda")
    out, err = run(x, s, 20)
    assert err == 0
    check(out, exact_scores(y, s), W, V)
    del x, buf
    torch.cuda.empty_cache()


def test_one_row_for_all_beams():
    x, s = make(1, 1, 999, FP, seed=13)
    s = torch.tensor([[-1.0, -2.5, -0.3]], device="cuda")
    out, err = run(x.expand(3, 999), s, 9)
    assert err == 0
    check(out, exact_scores(x.expand(3, 999), s), 3, 999)


def test_in_place_and_again():
    x, s = make(4, 8, 5003, BF, seed=14)
    done = torch.zeros(4, 8, dtype=torch.bool, device="cuda")
    done[1, 2] = True
    first, _ = run(x, s, finished=done, end_token=5)
    ws = mla.beam_workspace(4, 8, 5003)
    for _ in range(3):
        again, err = run(x, s, ws=ws, finished=done, end_token=5)
        assert err == 0 and all(torch.equal(a, b) for a, b in zip(first, again))
    s2, d2 = s.clone(), done.clone()
    out, _ = run(x, s2, ws=ws, finished=d2, end_token=5, scores_out=s2, finished_out=d2)
    assert out[2] is s2 and out[3] is d2
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    with pytest.raises(mla.MlaError):
        run(x, s, 4, ws=ws, scores_out=s.view(-1)[:16].view(4, 4))


def test_captured_and_two_workspaces():
    x, s = make(2, 4, 30001, BF, seed=15)
    y, t = make(2, 4, 30001, BF, seed=16)
    want = [run(a, b, 4)[0] for a, b in ((x, s), (y, t))]
    a, b = x.clone(), s.clone()
    ws = mla.beam_workspace(2, 4, 30001)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mla.mla_beam_select(a, b, 4, workspace_t=ws)
    for p, q, w in ((x, s, want[0]), (y, t, want[1]), (x, s, want[0])):
        a.copy_(p), b.copy_(q)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out[:3], w[:3]))
    # two at once, on streams and workspaces of their own
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(5):
        for k, (p, q) in enumerate(((x, s), (y, t))):
            got[k].append(mla.mla_beam_select(p, q, 4, stream=streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for o in got[k]:
            assert all(torch.equal(u, v) for u, v in zip(o[:3], want[k][:3]))


@pytest.mark.parametrize("B,W,V", [(64, 4, 700), (300, 2, 3001), (7, 8, 30000)])
def test_selections_right_behind_one_another(B, W, V):
    # each call's kernels start while the last one's run, and find its scores and flags
    x, s = make(B, W, V, BF, seed=18)
    done = torch.zeros(B, W, dtype=torch.bool, device="cuda")
    ws = mla.beam_workspace(B, W, V)
    s1, d1 = s.clone(), done.clone()
    for _ in range(40):
        mla.mla_beam_select(x, s1, finished=d1, end_token=3, scores_out=s1, finished_out=d1,
                            workspace_t=ws)
        torch.cuda.synchronize()
    s2, d2 = s.clone(), done.clone()
    torch.cuda.synchronize()
    for _ in range(40):
        mla.mla_beam_select(x, s2, finished=d2, end_token=3, scores_out=s2, finished_out=d2,
                            workspace_t=ws)
    torch.cuda.synchronize()
    assert torch.equal(s1, s2) and torch.equal(d1, d2)
    s3, d3 = s.clone(), done.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for _ in range(20):
            mla.mla_beam_select(x, s3, finished=d3, end_token=3, scores_out=s3, finished_out=d3,
                                workspace_t=ws)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(s1, s3) and torch.equal(d1, d3)
    assert mla.mla_read_device_error(ws) == 0


def test_no_requests_and_refusals():
    x, s = make(2, 4, 100, BF, seed=17)
    out = mla.mla_beam_select(x[:0], s[:0], 4)
    assert [t.shape for t in out[:3]] == [(0, 4)] * 3
    ws = mla.beam_workspace(2, 4, 100)
    kw = dict(workspace_t=ws)
    for bad in (dict(num_select=0), dict(num_select=33), dict(finished=s > 0, end_token=-1),
                dict(end_token=100), dict(finished=(s > 0)[:1], end_token=1),
                dict(finished=s, end_token=1), dict(tokens=torch.empty(2, 3, device="cuda").int()),
                dict(scores_out=torch.empty(2, 4, device="cuda").double())):
        with pytest.raises((ValueError, mla.MlaError)):
            mla.mla_beam_select(x, s, **bad, **kw)
    for logits, scores in ((x[:6], s), (x.double(), s), (x.t(), s), (x.cpu(), s), (x, s.double()),
                           (x, s.t()), (x, s.cpu()), (x.view(2, 4, 100), s), (x[:, :0], s)):
        with pytest.raises((ValueError, mla.MlaError)):
            mla.mla_beam_select(logits, scores, **kw)
    with pytest.raises(mla.MlaError):
        mla.mla_beam_select(x, s, workspace_t=ws[:mla.MLA_WORKSPACE_HEADER_BYTES])
