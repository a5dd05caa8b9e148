"""Host: what overlaps is refused.  Outputs overlap no input, no other output and no
workspace, but for the pairs that a call takes in place."""
import pytest
import torch

from test_beam_host import BUF, FAR, INVALID, DEVICE, lib, select  # noqa: F401

# (with a device what is not refused would run, on addresses that are none)
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="has a device")

READY = (DEVICE, -7)    # every check is passed

# two requests of four beams, bf16 rows of 1000, 2000 bytes apart; eight selected of each
SELECT = dict(logits=BUF, scores=BUF + FAR, finished=BUF + 7 * FAR, tokens=BUF + 2 * FAR,
              parents=BUF + 3 * FAR, scores_out=BUF + 4 * FAR, finished_out=BUF + 5 * FAR,
              workspace=BUF + 6 * FAR)
SIZE = dict(logits=16000, scores=32, finished=8, tokens=64, parents=64, scores_out=64,
            finished_out=16, workspace=16384)


def pairs(sizes, outputs, inputs, allowed=()):
    names = [(a, b) for i, a in enumerate(outputs) for b in [*outputs[i + 1:], *inputs]]
    return [(a, b, d) for a, b in names if (a, b) not in allowed
            for d in ("same", "first", "last") if sizes[a] and sizes[b]]


def placed(at, sizes, a, b, how):
    """The address of a that gives it b's place, b's first bytes or b's last ones."""
    return at[b] + {"same": 0, "first": 4 - sizes[a], "last": sizes[b] - 4}[how]


@pytest.mark.parametrize("a,b,how", pairs(
    SIZE, ["tokens", "parents", "scores_out", "finished_out"], ["logits", "scores", "finished"]))
def test_select(lib, a, b, how):    # noqa: F811
    assert select(lib, **{**SELECT, "num_select": 8, a: placed(SELECT, SIZE, a, b, how)}) == INVALID


@pytest.mark.parametrize("a", ["logits", "scores", "finished", "tokens", "parents", "scores_out",
                               "finished_out"])
def test_select_workspace(lib, a):  # noqa: F811
    for at in (SELECT["workspace"] + 2048, SELECT["workspace"] + 4 - SIZE[a]):
        assert select(lib, **{**SELECT, "num_select": 8, a: at}) == INVALID
    # behind what the call needs of it
    assert select(lib, **{**SELECT, "num_select": 8, a: SELECT["workspace"] + (1 << 20)}) in READY


def test_select_side_by_side(lib):  # noqa: F811
    kw = dict(SELECT, num_select=8)
    assert select(lib, **kw) in READY
    assert select(lib, **dict(kw, parents=kw["tokens"] + 64, scores_out=kw["tokens"] + 128,
                              finished_out=kw["tokens"] + 192)) in READY
    # between the logits' rows, and behind the last
    for at in (BUF + 2000, BUF + 7 * 4096 + 2000, BUF + 3 * 4096 - 64):
        assert select(lib, **dict(kw, row_stride=2048, tokens=at)) in READY
    for at in (BUF + 1999 // 4 * 4, BUF + 3 * 4096 - 60, BUF + 3 * 4096, BUF + 7 * 4096 + 1996):
        assert select(lib, **dict(kw, row_stride=2048, tokens=at)) == INVALID
    # one row for all
    assert select(lib, **dict(kw, row_stride=0, tokens=BUF + 2000)) in READY
    assert select(lib, **dict(kw, row_stride=0, tokens=BUF + 1996)) == INVALID
    # in place, and in place over the other one's place
    four = dict(SELECT, num_select=4)
    assert select(lib, **dict(four, scores_out=four["scores"], finished_out=four["finished"])) in READY
    assert select(lib, **dict(four, scores_out=four["scores"], tokens=four["scores"])) == INVALID
    assert select(lib, **dict(four, scores=BUF, scores_out=BUF)) == INVALID
    assert select(lib, **dict(four, finished=BUF + FAR, finished_out=BUF + FAR)) == INVALID
