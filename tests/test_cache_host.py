"""Host-side checks of the cache entry points that need no GPU: bad arguments
are refused before anything is enqueued."""
import ctypes
import os
import shutil

import pytest
import torch

from split_kv_mla_gb300 import build as mla_build
from split_kv_mla_gb300 import mla

BUF = 0x10000000   # a 256-byte aligned address that no refused call touches
WS = mla.MLA_WORKSPACE_HEADER_BYTES
INVALID, SHAPE, MISALIGNED, SMALL, DEVICE = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mla_build.LIB):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("library not built and nvcc not available")
        mla_build.build()
    return mla.load()


def append(lib, **kw):
    a = dict(kv=BUF, kv_stride=576, kv_weight=BUF, kv_norm_cols=512, slots=BUF, pool=BUF,
             pool_rows=64, row_bytes=576, kv_scale=0.03125, q=BUF, q_token_stride=16 * 192,
             q_head_stride=192, q_weight=None, q_norm=0, q_cols=192, q_nope=BUF, q_pe=BUF,
             positions=BUF, cos_sin=BUF, max_positions=128, half_split=0, eps=1e-6, num_tokens=4,
             num_heads=16, workspace=BUF, workspace_bytes=WS, stream=None)
    a.update(kw)
    return lib.mla_cache_append(*a.values())


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(num_tokens=-1)), (INVALID, dict(num_heads=-1)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))),
    (INVALID, dict(kv_scale=0.0)), (INVALID, dict(kv_scale=float("inf"))),
    (INVALID, dict(kv_scale=1e-42)),   # its reciprocal is no finite fp32 number
    (SHAPE, dict(row_bytes=640)), (SHAPE, dict(kv_norm_cols=64)),
    (SHAPE, dict(row_bytes=512)),   # 512 columns normed of a 512-byte row is fine, 448 too
    (SHAPE, dict(q_cols=96)), (SHAPE, dict(q_cols=0)), (SHAPE, dict(q_cols=640)),
    (SHAPE, dict(num_heads=129)), (INVALID, dict(num_heads=0)), (INVALID, dict(q=None)),
    (INVALID, dict(positions=None)), (INVALID, dict(cos_sin=None)),
    (INVALID, dict(max_positions=0)), (INVALID, dict(slots=None)), (INVALID, dict(pool=None)),
    (INVALID, dict(pool_rows=0)), (INVALID, dict(q_pe=None)), (INVALID, dict(q_nope=None)),
    (INVALID, dict(workspace=None)),
    (MISALIGNED, dict(kv=BUF + 8)), (MISALIGNED, dict(kv_stride=580)),
    (MISALIGNED, dict(kv_weight=BUF + 2)), (MISALIGNED, dict(pool=BUF + 4)),
    (MISALIGNED, dict(q=BUF + 2)), (MISALIGNED, dict(q_token_stride=3001)),
    (MISALIGNED, dict(q_head_stride=196)), (MISALIGNED, dict(q_nope=BUF + 8)),
    (MISALIGNED, dict(q_pe=BUF + 8)), (MISALIGNED, dict(cos_sin=BUF + 8)),
    (MISALIGNED, dict(workspace=BUF + 16)), (SMALL, dict(workspace_bytes=WS - 1)),
    (0, dict(num_tokens=0)), (0, dict(num_tokens=0, positions=None, workspace=None))])
def test_append_refusals(lib, want, kw):
    if kw == dict(row_bytes=512):
        kw = dict(row_bytes=512, kv_norm_cols=500)
    assert append(lib, **kw) == want


def fork(lib, **kw):
    a = dict(pool=BUF, pool_rows=64, row_bytes=576, kv_indices=BUF, num_indices=10,
             kv_indptr=BUF, num_parents=2, parents=BUF, keep=BUF, child_indptr=BUF,
             num_children=3, fresh=BUF, num_fresh=5, fresh_indptr=BUF, table=BUF, total=12,
             workspace=BUF, workspace_bytes=WS, stream=None)
    a.update(kw)
    return lib.mla_cache_fork(*a.values())


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(num_parents=-1)), (INVALID, dict(num_children=-1)),
    (INVALID, dict(num_indices=-1)), (INVALID, dict(num_fresh=-1)), (INVALID, dict(total=-1)),
    (SHAPE, dict(row_bytes=64)), (SHAPE, dict(total=1 << 31)),
    (INVALID, dict(pool=None)), (INVALID, dict(pool_rows=0)), (INVALID, dict(kv_indices=None)),
    (INVALID, dict(kv_indptr=None)), (INVALID, dict(parents=None)), (INVALID, dict(keep=None)),
    (INVALID, dict(child_indptr=None)), (INVALID, dict(fresh=None)),
    (INVALID, dict(fresh_indptr=None)), (INVALID, dict(table=None)),
    (INVALID, dict(workspace=None)), (MISALIGNED, dict(pool=BUF + 8)),
    (MISALIGNED, dict(workspace=BUF + 8)), (SMALL, dict(workspace_bytes=0)),
    (0, dict(num_children=0)), (0, dict(total=0))])
def test_fork_refusals(lib, want, kw):
    assert fork(lib, **kw) == want


def compact(lib, **kw):
    a = dict(pool=BUF, pool_rows=64, row_bytes=576, kv_indices=BUF, num_indices=10,
             new_indices=BUF, live=BUF, workspace=BUF, workspace_bytes=1 << 20, stream=None)
    a.update(kw)
    return lib.mla_cache_compact(*a.values())


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(num_indices=-1)), (INVALID, dict(pool_rows=0)), (SHAPE, dict(row_bytes=577)),
    (SHAPE, dict(pool_rows=1 << 31)), (SHAPE, dict(num_indices=1 << 31)),
    (INVALID, dict(pool=None)), (INVALID, dict(live=None)), (INVALID, dict(kv_indices=None)),
    (INVALID, dict(new_indices=None)), (INVALID, dict(workspace=None)),
    (MISALIGNED, dict(pool=BUF + 4)), (MISALIGNED, dict(workspace=BUF + 128)),
    (SMALL, dict(workspace_bytes=WS - 1)), (SMALL, dict(workspace_bytes=WS))])
def test_compact_refusals(lib, want, kw):
    assert compact(lib, **kw) == want


def test_compact_workspace_bytes(lib):
    size = lib.mla_cache_compact_workspace_bytes
    assert size(0) == size(-5) == size(1 << 31) == 0
    last = 0
    for n in (1, 31, 32, 8192, 8193, 100000, 1 << 20, (1 << 31) - 1):
        got = size(n)
        # the bitmap and its ranks at 32 slots a word, and a hole and a tail row each
        assert got >= WS + 2 * 4 * -(-n // 32) + 2 * 4 * (n // 2) and got >= last
        assert got % 256 == 0
        last = got


def test_binding_refusals():
    z = torch.zeros
    pool = z(8, 576, dtype=torch.uint8)
    i = z(4, dtype=torch.int32)
    with pytest.raises(ValueError):   # no CUDA tensors
        mla.mla_cache_compact(pool, i)
    with pytest.raises(ValueError):
        mla.mla_cache_fork(pool, i, i, i, i, i, 4, i, i)
    with pytest.raises(ValueError):
        mla.mla_cache_append(z(4, 576, dtype=torch.bfloat16), i, pool, i, z(8, 64))
    with pytest.raises(ValueError):   # neither rows nor queries
        mla.mla_cache_append(None, None, None, i, z(8, 64))
    with pytest.raises(ValueError):   # two bytes an element
        mla.mla_cache_compact(z(8, 288, dtype=torch.bfloat16), i)
    with pytest.raises(ValueError):   # rows apart
        mla.mla_cache_compact(z(8, 600, dtype=torch.uint8)[:, :576], i)


def test_no_device_is_an_error(lib):
    if torch.cuda.is_available():
        pytest.skip("has a device")
    for call in (append, fork):
        assert call(lib) in (DEVICE, -7)
    assert compact(lib) in (DEVICE, -7)
    assert ctypes.c_int(append(lib)).value != 0
