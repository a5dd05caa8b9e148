"""Host-side checks of the calls between two decode steps that need no GPU: bad
arguments are refused before anything is enqueued."""
import os
import shutil

import pytest
import torch

from split_kv_mla_gb300 import build as mla_build
from split_kv_mla_gb300 import mla

BUF = 0x10000000   # a 256-byte aligned address that no refused call touches
FAR = 1 << 32      # apart by more than any of the calls' buffers
WS = mla.MLA_WORKSPACE_HEADER_BYTES
INVALID, SHAPE, MISALIGNED, SMALL, DEVICE = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mla_build.LIB):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("library not built and nvcc not available")
        mla_build.build()
    return mla.load()


def select(lib, **kw):
    a = dict(logits=BUF, dtype=0, row_stride=1000, scores=BUF + FAR, finished=None, batch=2,
             beams=4, vocab=1000, num_select=4, end_token=3, tokens=BUF + 2 * FAR,
             parents=BUF + 3 * FAR, scores_out=BUF + 4 * FAR, finished_out=BUF + 5 * FAR,
             workspace=BUF + 6 * FAR, workspace_bytes=1 << 20, stream=None)
    a.update(kw)
    return lib.mla_beam_select(*a.values())


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(batch=-1)), (INVALID, dict(beams=0)), (INVALID, dict(vocab=0)),
    (INVALID, dict(num_select=0)), (INVALID, dict(dtype=3)), (INVALID, dict(dtype=-1)),
    (INVALID, dict(end_token=-2)), (INVALID, dict(end_token=1000)),
    (INVALID, dict(finished=BUF, end_token=-1)), (SHAPE, dict(num_select=33)),
    (SHAPE, dict(beams=33)), (SHAPE, dict(vocab=(1 << 20) + 1)), (SHAPE, dict(batch=65536)),
    (INVALID, dict(logits=None)), (INVALID, dict(scores=None)), (INVALID, dict(tokens=None)),
    (INVALID, dict(parents=None)), (INVALID, dict(scores_out=None)),
    (INVALID, dict(row_stride=-1)), (MISALIGNED, dict(logits=BUF + 1)),
    (MISALIGNED, dict(logits=BUF + 2, dtype=1)), (MISALIGNED, dict(workspace=BUF + 16)),
    (INVALID, dict(workspace=None)), (SMALL, dict(workspace_bytes=WS)),
    # in place only entry by entry
    (INVALID, dict(scores_out=BUF + FAR + 4)), (INVALID, dict(scores_out=BUF + FAR, num_select=3)),
    (INVALID, dict(finished=BUF, finished_out=BUF, num_select=8)),
    (INVALID, dict(finished=BUF, finished_out=BUF + 1)),
    (0, dict(batch=0)), (0, dict(batch=0, logits=None, workspace=None))])
def test_select_refusals(lib, want, kw):
    assert select(lib, **kw) == want


def test_select_workspace_bytes(lib):
    size = lib.mla_beam_select_workspace_bytes
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 33, 5), (65536, 1, 5), (1, 1, (1 << 20) + 1)):
        assert size(*bad) == 0
    for B, W, V in ((1, 1, 1), (1, 4, 32000), (64, 8, 131072), (3, 5, 257), (65535, 32, 1 << 20)):
        rows = B * W
        # a maximum of each 256 columns, and of each 1024 a maximum and a sum
        need = WS + rows * 4 * -(-V // 256) + rows * 8 * -(-V // 1024)
        # (or, of small calls, as many of fewer columns as the SMs take at a time)
        assert need <= size(B, W, V) <= need + 8 * 2 * 152 * 64 + 512
        assert size(B, W, V) % 256 == 0


def reorder(lib, **kw):
    a = dict(state=BUF, state_stride=64, num_parents=4, row_bytes=64, elem_bytes=4,
             parents=BUF + FAR, num_rows=4, lens=None, tokens=None, out=BUF + 2 * FAR, out_stride=64,
             out_lens=None, workspace=BUF + 3 * FAR, workspace_bytes=WS, stream=None)
    a.update(kw)
    return lib.mla_beam_reorder(*a.values())


LENS = dict(lens=BUF + 4 * FAR)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(num_parents=-1)), (INVALID, dict(num_rows=-1)), (INVALID, dict(row_bytes=-4)),
    (INVALID, dict(state_stride=-64)), (INVALID, dict(out_stride=-64)),
    (SHAPE, dict(elem_bytes=3)), (SHAPE, dict(elem_bytes=0)), (SHAPE, dict(elem_bytes=16)),
    (SHAPE, dict(row_bytes=62)), (SHAPE, dict(row_bytes=1 << 40, elem_bytes=4)),
    (INVALID, dict(tokens=BUF)), (INVALID, dict(out_lens=BUF)),
    (INVALID, dict(out_lens=BUF + 4 * FAR, **LENS)),
    (SHAPE, dict(tokens=BUF + 5 * FAR, elem_bytes=2, **LENS)),
    (MISALIGNED, dict(tokens=BUF + 5 * FAR, out=BUF + 2 * FAR + 2, **LENS)),
    (MISALIGNED, dict(tokens=BUF + 5 * FAR, out_stride=66, **LENS)),
    (INVALID, dict(parents=None)), (INVALID, dict(state=None)), (INVALID, dict(out=None)),
    (INVALID, dict(out_stride=60)), (INVALID, dict(workspace=None)),
    (MISALIGNED, dict(workspace=BUF + 8)), (SMALL, dict(workspace_bytes=WS - 1)),
    # rows that overlap: the same, shifted, of another stride, the last byte
    (INVALID, dict(out=BUF)), (INVALID, dict(out=BUF + 128)), (INVALID, dict(out=BUF + 255)),
    (INVALID, dict(out=BUF - 255)), (INVALID, dict(out=BUF + 64, state_stride=128, out_stride=64)),
    (INVALID, dict(out=BUF + 63, state_stride=128, out_stride=128)),
    (INVALID, dict(out=BUF + 65, state_stride=128, out_stride=128)),
    (INVALID, dict(out=BUF, state_stride=0)),
    # outputs over the other inputs and each other
    (INVALID, dict(out=BUF + FAR - 255)), (INVALID, dict(out=BUF + 4 * FAR, **LENS)),
    (INVALID, dict(tokens=BUF + 2 * FAR + 192, **LENS)),
    (INVALID, dict(out_lens=BUF + 4 * FAR + 12, **LENS)),
    (INVALID, dict(out_lens=BUF + FAR + 12, **LENS)),
    (INVALID, dict(out_lens=BUF + 2 * FAR - 12, **LENS)),
    (0, dict(num_rows=0)), (0, dict(num_rows=0, parents=None, state=None, out=None))])
def test_reorder_refusals(lib, want, kw):
    assert reorder(lib, **kw) == want


def extend(lib, **kw):
    a = dict(kv_indices=BUF, num_indices=100, kv_indptr=BUF + FAR, seq_lens=BUF + 2 * FAR,
             num_parents=4, parents=BUF + 3 * FAR, new_tokens=BUF + 4 * FAR, num_requests=6,
             free_slots=BUF + 5 * FAR, num_free=50, cursor=BUF + 6 * FAR, pool_rows=200,
             prefix_len=None, new_indices=BUF + 7 * FAR, total=150, new_indptr=BUF + 8 * FAR,
             new_lens=BUF + 9 * FAR, slots=BUF + 10 * FAR, positions=BUF + 11 * FAR, num_tokens=6,
             token_indptr=BUF + 12 * FAR, new_cursor=BUF + 13 * FAR, workspace=BUF + 14 * FAR,
             workspace_bytes=WS, stream=None)
    a.update(kw)
    return lib.mla_cache_extend(*a.values())


@pytest.mark.parametrize("want,kw", [
    *[(INVALID, {k: -1}) for k in ("num_indices", "num_parents", "num_requests", "num_free",
                                   "pool_rows", "total", "num_tokens")],
    *[(SHAPE, {k: 1 << 31}) for k in ("num_indices", "num_free", "pool_rows", "total",
                                      "num_tokens")],
    *[(INVALID, {k: None}) for k in ("kv_indices", "kv_indptr", "seq_lens", "cursor", "new_indices",
                                     "new_indptr", "new_lens", "slots", "positions", "token_indptr",
                                     "new_cursor", "workspace")],
    (INVALID, dict(parents=None)),   # six requests of four
    (MISALIGNED, dict(workspace=BUF + 8)), (SMALL, dict(workspace_bytes=0)),
    # outputs over inputs
    (INVALID, dict(new_indices=BUF)), (INVALID, dict(new_indices=BUF + 396)),
    (INVALID, dict(new_indptr=BUF + FAR)), (INVALID, dict(new_lens=BUF + 2 * FAR)),
    (INVALID, dict(new_lens=BUF + 3 * FAR + 20)), (INVALID, dict(slots=BUF + 5 * FAR + 196)),
    (INVALID, dict(token_indptr=BUF + 4 * FAR - 24)), (INVALID, dict(positions=BUF + 6 * FAR - 20)),
    (INVALID, dict(prefix_len=BUF + 13 * FAR))])
def test_extend_refusals(lib, want, kw):
    assert extend(lib, **kw) == want


def test_binding_refusals():
    z, i32 = torch.zeros, torch.int32
    i = z(4, dtype=i32)
    with pytest.raises(ValueError):   # no CUDA tensors
        mla.mla_beam_select(z(4, 10), z(1, 4))
    with pytest.raises(ValueError):
        mla.mla_beam_reorder(z(4, 10), i)
    with pytest.raises(ValueError):
        mla.mla_cache_extend(i, i, i[:3], i[:1], 4, 4, 100)
    ws = z(1 << 17, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_beam_select(z(4, 10), z(1, 4), workspace_t=ws)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_beam_reorder(z(4, 10), i, workspace_t=ws)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_cache_extend(i, i, i[:3], i[:1], 4, 4, 100, workspace_t=ws)
    with pytest.raises(ValueError, match="not supported"):
        mla.beam_workspace(1, 33, 100, device="cpu")


def test_no_device_is_an_error(lib):
    if torch.cuda.is_available():
        pytest.skip("has a device")
    for call in (select, reorder, extend):
        assert call(lib) in (DEVICE, -7)
    # what is allowed: the cursor in place, the last entries side by side
    assert extend(lib, new_cursor=BUF + 6 * FAR) in (DEVICE, -7)
    assert extend(lib, new_indices=BUF + 400) in (DEVICE, -7)
    assert select(lib, scores_out=BUF + FAR, finished=BUF, finished_out=BUF) in (DEVICE, -7)
    assert reorder(lib, out=BUF + 64, state_stride=128, out_stride=128) in (DEVICE, -7)
