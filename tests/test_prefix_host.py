"""Host-side checks of the shared-prefix decode that need no GPU: plans follow
from shapes alone, the partials fit for every length, bad arguments are refused
before anything is enqueued."""
import ctypes
import os
import shutil

import pytest
import torch

from split_kv_mla_gb300 import build as mla_build
from split_kv_mla_gb300 import mla

BUF = 0x10000000
INVALID, SHAPE, MISALIGNED, SMALL, DEVICE = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mla_build.LIB):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("library not built and nvcc not available")
        mla_build.build()
    return mla.load()


SHAPES = [(1, 1, 1, 1, 0), (1, 1, 16, 127, 5), (4, 1, 16, 1024, 130), (64, 1, 16, 8192, 16896),
          (8, 4, 16, 32001, 1200), (64, 1, 128, 32768, 32768), (64, 1, 128, 0, 100),
          (128, 4, 128, 100, 0), (3, 7, 5, 1 << 20, 10), (1, 1, 128, 131072, 0),
          (0, 1, 16, 100, 0), (65535, 1, 1, 300, 65535)]


@pytest.mark.parametrize("batch,q_len,heads,cap,total", SHAPES)
@pytest.mark.parametrize("sms", [1, 20, 152])
def test_plan_invariants(lib, batch, q_len, heads, cap, total, sms):
    p = mla.mla_prefix_decode_plan(batch, q_len, heads, cap, total, sms)
    rows = batch * q_len * heads
    blocks = -(-cap // 128)
    assert p.tiles == -(-rows // 64)
    assert (p.prefix_cap, p.sm_count) == (cap, sms)
    assert p.own.as_dict() == mla.mla_decode_plan(batch, q_len, heads, total, sms).as_dict()
    if cap == 0 or rows == 0:
        assert (p.ctas, p.parts) == (0, 0)
    else:
        assert 1 <= p.ctas <= sms and p.ctas <= p.tiles * blocks and 1 <= p.parts <= 256
    def up(x):
        return -(-x // 256) * 256
    ns, tiles = p.own.num_splits, p.tiles if p.parts else 0
    want = mla.MLA_WORKSPACE_HEADER_BYTES + sum(map(up, (
        rows * ns * 2048, rows * ns * 4, rows * p.parts * 2048, rows * p.parts * 4,
        blocks * 73728, blocks * 16, tiles * 73728, tiles * 256, tiles * 256)))
    assert p.workspace_bytes == want
    q = mla.mla_prefix_decode_plan(batch, q_len, heads, cap, total, sms)
    assert bytes(p) == bytes(q)


@pytest.mark.parametrize("batch,q_len,heads,cap,total", SHAPES)
def test_every_length_fits_the_planned_partials(lib, batch, q_len, heads, cap, total):
    # runs of (tile, block) pairs as the kernel deals them out: every pair once, a
    # tile's runs numbered 0, 1, ... below parts, whatever the length in use
    p = mla.mla_prefix_decode_plan(batch, q_len, heads, cap, total, 152)
    if p.parts == 0:
        return
    T = min(p.tiles, 300)
    most = -(-cap // 128)
    for blocks in sorted({1, 2, 3, 7, most // 3 + 1, most - 1, most} & set(range(1, most + 1))):
        U = p.tiles * blocks
        G = min(p.ctas, U)
        def first(u):
            return ((u + 1) * G - 1) // U
        for t in range(T):
            cut = [g * U // G for g in range(first(t * blocks), first((t + 1) * blocks - 1) + 2)]
            assert cut[0] <= t * blocks < cut[1]
            assert cut[-2] < (t + 1) * blocks <= cut[-1]
            assert len(cut) - 1 <= p.parts
            assert all(b > a for a, b in zip(cut, cut[1:]))


def test_plan_refusals(lib):
    for bad in [(-1, 1, 16, 10, 10, 152), (1, 0, 16, 10, 10, 152), (1, 1, 0, 10, 10, 152),
                (1, 1, 129, 10, 10, 152), (65536, 1, 1, 10, 10, 152), (1, 1, 16, -1, 10, 152),
                (1, 1, 16, (1 << 30) + 1, 10, 152), (1, 1, 16, 10, -1, 152), (1, 1, 16, 10, 10, 0),
                (65535, 1024, 128, 10, 10, 152)]:
        with pytest.raises(mla.MlaError):
            mla.mla_prefix_decode_plan(*bad)
    assert lib.mla_prefix_decode_plan(1, 1, 16, 10, 10, 152, None) == INVALID


def call(lib, plan, **kw):
    a = dict(plan=ctypes.byref(plan) if plan is not None else None, q_lat=BUF, q_pe=BUF, pool=BUF,
             pool_rows=64, prefix_indices=BUF, prefix_len=BUF, seq_lens=BUF, kv_indices=BUF,
             kv_indptr=BUF, batch=2, q_len=1, num_heads=16, scale=0.04, kv_scale=0.03, o=BUF,
             lse=BUF, workspace=BUF, workspace_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.mla_prefix_decode(*a.values())


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(batch=3)), (INVALID, dict(q_len=2)), (INVALID, dict(num_heads=8)),
    (INVALID, dict(q_lat=None)), (INVALID, dict(q_pe=None)), (INVALID, dict(pool=None)),
    (INVALID, dict(pool_rows=0)), (INVALID, dict(prefix_indices=None)),
    (INVALID, dict(seq_lens=None)), (INVALID, dict(kv_indices=None)),
    (INVALID, dict(kv_indptr=None)), (INVALID, dict(o=None)), (INVALID, dict(workspace=None)),
    (INVALID, dict(scale=float("nan"))), (INVALID, dict(kv_scale=float("inf"))),
    (MISALIGNED, dict(q_lat=BUF + 2)), (MISALIGNED, dict(q_pe=BUF + 8)),
    (MISALIGNED, dict(pool=BUF + 4)), (MISALIGNED, dict(o=BUF + 8)),
    (MISALIGNED, dict(workspace=BUF + 64)), (SMALL, dict(workspace_bytes=70000))])
def test_call_refusals(lib, want, kw):
    p = mla.mla_prefix_decode_plan(2, 1, 16, 1000, 100, 152)
    assert call(lib, p, **kw) == want


def test_tampered_plans_are_refused(lib):
    good = mla.mla_prefix_decode_plan(2, 1, 16, 1000, 100, 152)
    assert call(lib, None) == INVALID
    for field, value in [("tiles", 2), ("ctas", 0), ("ctas", -3), ("parts", 0), ("parts", 300),
                         ("workspace_bytes", 1 << 20), ("prefix_cap", 5000), ("prefix_cap", -1),
                         ("prefix_cap", 0)]:
        p = mla.mla_prefix_plan_t.from_buffer_copy(good)
        setattr(p, field, value)
        assert call(lib, p) == INVALID, field
    for field, value in [("num_splits", 3), ("grid_x", 9), ("variant", 1), ("merge_cluster", 2),
                         ("workspace_bytes", 4), ("d_v", 448), ("total_keys", -1)]:
        p = mla.mla_prefix_plan_t.from_buffer_copy(good)
        setattr(p.own, field, value)
        assert call(lib, p) == INVALID, field


def test_no_device_is_an_error(lib):
    if torch.cuda.is_available():
        pytest.skip("has a device")
    p = mla.mla_prefix_decode_plan(2, 1, 16, 1000, 100, 152)
    assert call(lib, p) in (DEVICE, -7)
    empty = mla.mla_prefix_decode_plan(0, 1, 16, 1000, 0, 152)
    assert call(lib, empty, batch=0) == 0


def test_binding_refusals():
    p = mla.mla_prefix_decode_plan(2, 1, 16, 4, 4, 152)
    z = torch.zeros
    i = z(4, dtype=torch.int32)
    with pytest.raises(ValueError):   # no CUDA tensors
        mla.mla_prefix_decode(p, z(2, 16, 512, dtype=torch.bfloat16),
                              z(2, 16, 64, dtype=torch.bfloat16), z(8, 576, dtype=torch.uint8),
                              i, i[:2], i, i[:3], 0.04, 0.03)
