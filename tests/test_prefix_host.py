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


def workspace_bytes(p):
    """The plan's workspace from its other fields."""
    def up(x):
        return -(-x // 256) * 256
    rows = p.own.batch * p.own.q_len * p.own.num_heads
    blocks = -(-p.prefix_cap // 128)
    own = 0 if p.joined or p.own.total_keys == 0 else rows * p.own.num_splits
    if p.joined:
        blocks += p.own.total_keys // 128 + p.own.batch
    slots = 0 if p.ctas == 0 else p.ctas if p.splits else p.ctas + p.tiles
    tiles = p.tiles if p.ctas else 0
    return mla.MLA_WORKSPACE_HEADER_BYTES + sum(map(up, (
        own * 2048, own * 4, slots * 64 * 2048, slots * 64 * 4, blocks * 73728, blocks * 32,
        tiles * 73728, tiles * 256, tiles * 256, (tiles + 1) * 8 if tiles else 0)))


@pytest.mark.parametrize("batch,q_len,heads,cap,total", SHAPES)
@pytest.mark.parametrize("sms", [1, 20, 152])
def test_plan_invariants(lib, batch, q_len, heads, cap, total, sms):
    p = mla.mla_prefix_decode_plan(batch, q_len, heads, cap, total, sms)
    rows = batch * q_len * heads
    assert p.tiles == -(-rows // 64)
    assert (p.prefix_cap, p.sm_count) == (cap, sms)
    assert p.own.as_dict() == mla.mla_decode_plan(batch, q_len, heads, total, sms).as_dict()
    if cap == 0 or rows == 0:
        assert (p.ctas, p.splits, p.joined) == (0, 0, 0)
    else:
        assert 1 <= p.ctas <= sms and p.ctas == (p.tiles * p.splits or p.ctas)
        assert p.joined in (0, 1) and not (p.joined and total == 0)
    assert p.workspace_bytes == workspace_bytes(p)
    q = mla.mla_prefix_decode_plan(batch, q_len, heads, cap, total, sms)
    assert bytes(p) == bytes(q)


def test_plan_choices(lib):
    # short own keys join the tiles, long ones go through the split kernel (measured);
    # many tiles are cut into equal runs, few into equal parts
    def of(*a):
        p = mla.mla_prefix_decode_plan(*a, 152)
        return p.ctas, p.splits, p.joined
    assert of(64, 1, 16, 8192, 64 * 264) == (144, 9, 1)
    assert of(64, 1, 16, 8192, 64 * 8192)[2] == 0
    assert of(64, 1, 128, 32768, 64 * 512) == (152, 0, 1)
    assert of(8, 4, 16, 32001, 8 * 150) == (152, 19, 1)


@pytest.mark.parametrize("seed", range(12))
def test_runs_cover_every_block_once(seed):
    # blocks of tiles (some empty) as the kernel deals them out: each once, in order,
    # and no two runs share a slot
    import random
    rng = random.Random(seed)
    tiles = rng.choice([1, 2, 5, 16, 130, 700])
    nb = [rng.choice([0, 1, 3, 64, rng.randrange(300)]) for _ in range(tiles)]
    start = [0]
    for n in nb:
        start.append(start[-1] + n)
    seen, slots = [], set()
    splits = rng.choice([0, 1, 7, 19])
    ctas = tiles * splits or rng.choice([1, 2, 37, 152])
    U = start[-1]
    G = min(ctas, U)
    runs_of = [[] for _ in range(tiles)]
    for g in range(ctas):
        if splits:
            t, s = divmod(g, splits)
            x0, x1 = nb[t] * s // splits, nb[t] * (s + 1) // splits
            runs = [(t, x0, x1, g)] if x1 > x0 else []
        else:
            runs = []
            u, end = (g * U // G, (g + 1) * U // G) if g < G else (0, 0)
            while u < end:
                t = max(i for i in range(tiles) if start[i] <= u and nb[i] > 0)
                x0 = u - start[t]
                x1 = min(nb[t], x0 + end - u)
                runs.append((t, x0, x1, g + t))
                u += x1 - x0
        for t, x0, x1, slot in runs:
            seen += [(t, x) for x in range(x0, x1)]
            assert slot not in slots
            slots.add(slot)
            runs_of[t].append(slot)
    assert sorted(seen) == [(t, x) for t in range(tiles) for x in range(nb[t])]
    for t in range(tiles):   # where the merge looks
        if nb[t] == 0:
            assert runs_of[t] == []
        elif splits:
            want = [t * splits + s for s in range(splits)
                    if nb[t] * s // splits < nb[t] * (s + 1) // splits]
            assert runs_of[t] == want
        else:
            g0 = ((start[t] + 1) * G - 1) // U
            g1 = (start[t + 1] * G - 1) // U
            assert runs_of[t] == list(range(g0 + t, g1 + t + 1))
            assert max(runs_of[t]) < ctas + tiles


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
    for field, value in [("tiles", 2), ("ctas", 0), ("ctas", -3), ("ctas", 300), ("splits", -1),
                         ("splits", 300), ("splits", good.splits + 1), ("joined", 2),
                         ("joined", 1 - good.joined), ("workspace_bytes", 1 << 20),
                         ("prefix_cap", 5000), ("prefix_cap", -1), ("prefix_cap", 0)]:
        p = mla.mla_prefix_plan_t.from_buffer_copy(good)
        setattr(p, field, value)
        if (p.ctas, p.splits) == (good.ctas, good.splits) or not good.splits:
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


def test_binding_refuses_other_objects():
    z = torch.zeros
    i = z(4, dtype=torch.int32)
    args = (z(2, 16, 512, dtype=torch.bfloat16), z(2, 16, 64, dtype=torch.bfloat16),
            z(8, 576, dtype=torch.uint8), i, i[:2], i, i[:3], 0.04, 0.03)
    ws = z(1 << 20, dtype=torch.uint8)
    with pytest.raises(TypeError):    # the plan of the plain decode
        mla.mla_prefix_decode(mla.mla_plan_t(), *args)
    with pytest.raises(TypeError):
        mla.mla_prefix_decode(None, *args)
    p = mla.mla_prefix_decode_plan(2, 1, 16, 4, 4, 152)
    for k in range(7):                # neither a list nor nothing is a tensor
        for other in ([1, 2], None):
            with pytest.raises(ValueError):
                mla.mla_prefix_decode(p, *args[:k], other, *args[k + 1:], workspace_t=ws)


def test_binding_refusals():
    p = mla.mla_prefix_decode_plan(2, 1, 16, 4, 4, 152)
    z = torch.zeros
    i = z(4, dtype=torch.int32)
    with pytest.raises(ValueError):   # no CUDA tensors
        mla.mla_prefix_decode(p, z(2, 16, 512, dtype=torch.bfloat16),
                              z(2, 16, 64, dtype=torch.bfloat16), z(8, 576, dtype=torch.uint8),
                              i, i[:2], i, i[:3], 0.04, 0.03)
