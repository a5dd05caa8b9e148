"""Host: what overlaps is refused.  Outputs overlap no input, no other output and no
workspace, but for the pairs that a call takes in place."""
import pytest
import torch

from test_beam_host import BUF, FAR, INVALID, DEVICE, WS, extend, lib, reorder, select  # noqa: F401

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


# the entries of the call's defaults, of four bytes; six requests of four, six tokens
EXTEND = dict(kv_indices=BUF, kv_indptr=BUF + FAR, seq_lens=BUF + 2 * FAR, parents=BUF + 3 * FAR,
              new_tokens=BUF + 4 * FAR, free_slots=BUF + 5 * FAR, cursor=BUF + 6 * FAR,
              new_indices=BUF + 7 * FAR, new_indptr=BUF + 8 * FAR, new_lens=BUF + 9 * FAR,
              slots=BUF + 10 * FAR, positions=BUF + 11 * FAR, token_indptr=BUF + 12 * FAR,
              new_cursor=BUF + 13 * FAR, workspace=BUF + 14 * FAR, prefix_len=BUF + 15 * FAR)
ENTRIES = {k: 4 * n for k, n in dict(
    kv_indices=100, kv_indptr=5, seq_lens=4, parents=6, new_tokens=6, free_slots=50, cursor=1,
    prefix_len=1, new_indices=150, new_indptr=7, new_lens=6, slots=6, positions=6, token_indptr=7,
    new_cursor=1).items()}
EXTENDED = ["new_indices", "new_indptr", "new_lens", "slots", "positions", "token_indptr",
            "new_cursor"]


@pytest.mark.parametrize("a,b,how", pairs(
    ENTRIES, EXTENDED, [k for k in ENTRIES if k not in EXTENDED], [("new_cursor", "cursor")]))
def test_extend(lib, a, b, how):    # noqa: F811
    assert extend(lib, **{**EXTEND, a: placed(EXTEND, ENTRIES, a, b, how)}) == INVALID


@pytest.mark.parametrize("a", list(ENTRIES))
def test_extend_workspace(lib, a):  # noqa: F811
    at = EXTEND["workspace"]
    for x in (at, at + 4 - ENTRIES[a], at + WS - 4):
        assert extend(lib, **{**EXTEND, a: x}) == INVALID
    assert extend(lib, **{**EXTEND, a: at + WS}) in READY


def test_extend_side_by_side(lib):  # noqa: F811
    assert extend(lib, **EXTEND) in READY
    at, kw = BUF + 20 * FAR, dict(EXTEND)
    for name in EXTENDED:
        kw[name] = at
        at += ENTRIES[name]
    assert extend(lib, **kw) in READY
    assert extend(lib, **dict(kw, new_cursor=kw["cursor"])) in READY
    # what has no entries overlaps nothing
    none = dict(kw, num_tokens=0, slots=BUF, positions=BUF, total=0, new_indices=BUF)
    assert extend(lib, **none) in READY


# four rows of 64 bytes of four
REORDER = dict(state=BUF, parents=BUF + FAR, out=BUF + 2 * FAR, workspace=BUF + 3 * FAR,
               lens=BUF + 4 * FAR, tokens=BUF + 5 * FAR, out_lens=BUF + 6 * FAR)
ROWS = dict(state=256, parents=16, out=256, lens=16, tokens=16, out_lens=16)


@pytest.mark.parametrize("a,b,how", pairs(ROWS, ["out", "out_lens"],
                                          ["state", "parents", "lens", "tokens"]))
def test_reorder(lib, a, b, how):   # noqa: F811
    assert reorder(lib, **{**REORDER, a: placed(REORDER, ROWS, a, b, how)}) == INVALID


@pytest.mark.parametrize("a", list(ROWS))
def test_reorder_workspace(lib, a):     # noqa: F811
    at = REORDER["workspace"]
    for x in (at, at + 4 - ROWS[a], at + WS - 4):
        assert reorder(lib, **{**REORDER, a: x}) == INVALID
    assert reorder(lib, **{**REORDER, a: at + WS}) in READY


def test_reorder_side_by_side(lib):     # noqa: F811
    assert reorder(lib, **REORDER) in READY
    # between the rows of the state, and of out
    between = dict(REORDER, state_stride=128, out_stride=128)
    assert reorder(lib, **dict(between, out_lens=BUF + 64)) in READY
    assert reorder(lib, **dict(between, out_lens=BUF + 3 * 128 + 64)) in READY
    assert reorder(lib, **dict(between, out_lens=BUF + 60)) == INVALID
    assert reorder(lib, **dict(between, out_lens=BUF + 116)) == INVALID
    assert reorder(lib, **dict(between, out_lens=BUF + 3 * 128 + 60)) == INVALID
    # one row for all
    assert reorder(lib, **dict(REORDER, state_stride=0, out_lens=BUF + 64)) in READY
    assert reorder(lib, **dict(REORDER, num_parents=0, out_lens=BUF)) in READY
    # one list as parents and as lengths is as long as both
    same = dict(REORDER, lens=BUF + FAR, num_parents=2)
    assert reorder(lib, **same) in READY
    assert reorder(lib, **dict(same, out_lens=BUF + FAR + 12)) == INVALID
