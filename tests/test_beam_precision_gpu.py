"""GPU: the scores of rows in which one token has most of the mass, near 0.

With m a row's maximum and t the sum of e^(x - m) over its other logits, a score is
cum + (x - m) - ln(1 + t), rounded to fp32 (half a step, 2^-24 of its value).  What the
logarithm carries, in units of 2^-24 of it, is for t < 0.5 what t does:
- a term's exponent, in a segment of the row: 2.25 times its distance d from the segment's
  maximum (d and its product with log2 e are rounded, log2 e is off by a quarter).  Terms
  that count have d below 88: 198;
- 4 of the exponential, 4 of e^(the segment's maximum - m), 4 of log1p;
- an addition each, of at most 38 in a segment, and 32 in m's own, 16 and 6 over the segments.
And for t of 0.5 or more, where the logarithm is 0.4 and more, two and a half times what
1 + t does: 60 additions, 8 of the exponentials, 4 of ln, and 2.25 times the mean of d, which
is below 20 (more than e^-20 of 2^20 terms): 117.
Both are below 512: 2^-15 of the logarithm.  Terms below 2^-126 are none: 2^-106 for 2^20.
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


def reference(logits, scores):
    """float64: scores [B, W * V] and what they may be off by."""
    B, W = scores.shape
    x = logits.cpu().double()
    m, at = x.max(-1, keepdim=True)
    e = torch.exp(x - m)
    e.scatter_(1, at, 0.0)                   # (one of the maxima; the others are terms)
    ln = torch.log1p(e.sum(-1, keepdim=True))
    s = scores.cpu().double().view(-1, 1) + ((x - m) - ln)
    off = s.abs() * 2.0 ** -24 + ln * 2.0 ** -15 + 2.0 ** -106
    return s.view(B, -1), off.view(B, -1)


def check(logits, scores, K):
    B, W = scores.shape
    V = logits.shape[1]
    ws = mla.beam_workspace(B, W, V)
    tokens, parents, got, _ = (None if t is None else t.cpu() for t in mla.mla_beam_select(
        logits, scores, K, workspace_t=ws))
    assert mla.mla_read_device_error(ws) == 0
    want, off = reference(logits, scores)
    at = (parents.long() - torch.arange(B)[:, None] * W) * V + tokens.long()
    err = (got.double() - want.gather(1, at)).abs()
    limit = off.gather(1, at)
    assert bool((err <= limit).all()), float((err / limit).max())
    # and they are the best, in their order, as far as both are that exact
    top = want.topk(K)
    assert bool(((top.values - got.double()).abs() <= off.gather(1, top.indices)).all())
    return got


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("V", [7, 300, 4099, 32000, 100003])
@pytest.mark.parametrize("cum", [0.0, -1e-6, -0.01, -3.0])
def test_confident_rows(dtype, V, cum):
    g = torch.Generator().manual_seed(V)
    ahead = [0.0, 3.0, 6.0, 9.0, 12.0, 15.0, 18.0, 20.0, 24.0, 30.0, 40.0, 70.0]
    B, W = 3, len(ahead)
    x = torch.randn(B * W, V, generator=g)
    x.scatter_(1, torch.randint(0, V, (B * W, 1), generator=g), torch.tensor(ahead * B)[:, None])
    s = torch.full((B, W), cum)
    s[1] *= torch.rand(W, generator=g)
    s[2, ::2] = -0.5
    check(x.to(dtype).cuda(), s.cuda(), W)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("V", [2, 513, 50001])
def test_two_tokens_ahead(dtype, V):
    # in one segment and in two, equal and one step apart; and rows that start at odd places
    W = 6
    flat = torch.randn(W * (V + 1) + 1, generator=torch.Generator().manual_seed(V))
    x = flat.to(dtype).cuda()[1:].view(W, V + 1)[:, :V]
    for w, (a, b) in enumerate([(20, 20), (20, 19.875), (25, 12), (14, 14), (14, 13), (30, 30)]):
        x[w, V // 3], x[w, V - 1 - w % 2 * (V // 4)] = a, b
    check(x, torch.tensor([[0.0, 0.0, 0.0, -1e-4, -0.25, -20.0]]).cuda(), W)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_one_token_left(dtype):
    # nothing else has any mass: the score is the beam's own, to the bit
    W, V = 4, 5003
    x = torch.full((W, V), -math.inf, dtype=dtype, device="cuda")
    x[torch.arange(W), torch.tensor([0, 17, 2048, V - 1])] = torch.tensor(
        [0.0, -9.0, 400.0, 1e-3], dtype=dtype, device="cuda")
    s = torch.tensor([[-1e-7, -0.3, -1.5, -40.0]], device="cuda")
    got = check(x, s, W)
    assert torch.equal(got[0], s[0].cpu())


def exact_rows(dtype, level, seed):
    """Beams of 2^n equal logits and nothing else, so that their sums are exact, whose
    scores lie one or two fp32 steps from one another: (logits, scores, float64 scores of
    the beams' tokens)."""
    g = torch.Generator().manual_seed(seed)
    W, V = 8, 5003
    n = torch.randint(0, 11, (W,), generator=g)
    x = torch.full((W, V), -math.inf)
    for w in range(W):
        at = torch.randperm(V, generator=g)[:2 ** int(n[w])]
        x[w, at] = [0.0, -3.0, 13.5, 7.25][w % 4]
    step = 2.0 ** (math.floor(math.log2(-level)) - 23)
    apart = torch.randint(0, 3, (W,), generator=g).cumsum(0)[torch.randperm(W, generator=g)]
    s = (level + n.double() * math.log(2.0) - apart * step).float()
    return x.to(dtype), s.view(1, W), s.double() - n.double() * math.log(2.0)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("level", [-1.3, -7.7, -41.0, -97.5])
@pytest.mark.parametrize("seed", range(4))
def test_steps_between_beams(dtype, level, seed):
    """Before it is rounded such a score is off by less than 2^-32: the parts of cum - m - n ln 2
    below the first float, 2^-17 at most, and n times what ln 2 has below its first part,
    3.3e-4, are rounded three times each.  Scores that lie no nearer than that to the middle
    of two numbers come out as the rounded ones, and in their order."""
    x, s, score = exact_rows(dtype, level, seed)
    step = torch.exp2(torch.floor(torch.log2(-score)) - 23)
    middle = ((score / step) % 1 - 0.5).abs() * step
    assert bool((middle > 2.0 ** -31).all())    # (of these inputs)
    want = [(-float(score[w].float()), w, v) for w in range(x.shape[0])
            for v in (x[w] > -math.inf).nonzero()[:, 0].tolist()]
    want = sorted(want)[:32]
    tokens, parents, got, _ = mla.mla_beam_select(x.cuda(), s.cuda(), 32)
    n = len(want)
    assert list(zip(parents[0, :n].tolist(), tokens[0, :n].tolist())) == [(w, v) for _, w, v in want]
    assert got[0, :n].tolist() == [-a for a, _, _ in want]
    assert bool((tokens[0, n:] == -1).all())


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("V", [12, 4099])
@pytest.mark.parametrize("shift", [-45.0, 60.0, 777.0, -3000.0, 30000.0])
def test_scores_far_below_the_logits(dtype, V, shift):
    # (what a logit's size is does not matter: a score is a difference)
    g = torch.Generator().manual_seed(V)
    W = 16
    x = torch.randn(W, V, generator=g) * 3
    x[:, V // 2] = torch.linspace(8, 30, W)
    step = {FP: 0.0, HF: 2.0 ** -10, BF: 2.0 ** -7}[dtype] * abs(shift)   # kept apart by the type
    x = (x * max(1.0, step) + shift).to(dtype)
    for size in (0.0, 1e-8, 1e-7, 1e-6, 1e-5, 1e-4, 1e-3, 1e-2):
        s = -size * torch.rand(1, W, generator=g)
        check(x.cuda(), s.cuda(), W)
        check(x.cuda(), -s.cuda(), 2 * W)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("m", [27.25, 19.0, 61.0, 0.75])
def test_scores_of_half_a_step_of_the_maximum(dtype, m):
    # where cum - m rounds to a neighbour of m, one rounding must not follow another
    W, V = 32, 10
    g = torch.Generator().manual_seed(int(m))
    x = torch.randn(W, V, generator=g) * 0.4 + (m - 25)
    x[:, 3] = m
    half = 2.0 ** (math.floor(math.log2(m)) - 24)
    for lo, hi in ((0.98, 1.06), (0.5, 2.0)):
        s = -half * (lo + (hi - lo) * torch.rand(4, W, generator=g))
        check(x.repeat(4, 1).to(dtype).cuda(), s.cuda(), W)
