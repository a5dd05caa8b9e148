"""GPU: calls with ``stream=`` that allocate their own outputs and workspaces.

What a call allocates is zeroed on its stream and belongs to it: the current stream may
be far behind (the zeroing would come late) or ahead (it would hand the memory out
again while the call still runs).
"""
import pytest
import torch

from oracle import oracle
from split_kv_mla_gb300 import inputs as gen
from split_kv_mla_gb300 import mla

from gpu_util import compare, dense_to_cuda
from test_prefix_gpu import make, plan_of, to_cuda

pytestmark = pytest.mark.gpu

PAUSE = 100_000_000   # cycles, about 50 ms


@pytest.fixture(scope="module", autouse=True)
def _built():
    oracle.build()
    mla.load()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls():
    """name -> a call of its inputs that takes `stream` alone and returns its outputs."""
    s = make(1, 16, 900, [30, 700], seed=70)
    d, plan = to_cuda(s), plan_of(s)
    out = {"prefix": lambda **kw: mla.mla_prefix_decode(plan, **d, scale=s.own.scale,
                                                        kv_scale=s.own.kv_scale, **kw)}
    inp = gen.dense_inputs(2, 1, 16, [3000, 700], seed=71)
    dd = dense_to_cuda(inp)
    dplan = mla.mla_decode_plan(2, 1, 16, inp.total_keys, mla.sm_count())
    args = (dd["q_lat"], dd["q_pe"], dd["pool"], dd["seq_lens"], dd["kv_indices"],
            dd["kv_indptr"], inp.scale, inp.kv_scale)
    out["decode"] = lambda **kw: mla.mla_decode(dplan, *args, **kw)
    out["dcp"] = lambda **kw: mla.mla_decode_dcp(dplan, *args, None, 0, 1, **kw)
    sp = gen.sparse_extra_inputs(2, 16, 500, 64, 4000, 1000, seed=72)
    splan = mla.mla_sparse_decode_plan(2, 16, 500, mla.sm_count())
    xplan = mla.mla_sparse_decode_plan(2, 16, 500, mla.sm_count(), extra_topk=64)
    q = [t.cuda() for t in (sp.q_nope, sp.q_pe, sp.pool, sp.indices)]
    x = [t.cuda() for t in (sp.extra_pool, sp.extra_indices)]
    out["sparse"] = lambda **kw: mla.mla_sparse_decode(splan, *q, sp.scale, sp.kv_scale, **kw)
    out["extra"] = lambda **kw: mla.mla_sparse_decode_extra(xplan, *q, *x, sp.scale, sp.kv_scale,
                                                            **kw)
    g = torch.Generator(device="cuda").manual_seed(73)
    parts = torch.randn(300, 20, 512, generator=g, device="cuda")
    lses = torch.randn(300, 20, generator=g, device="cuda")
    out["reduce"] = lambda **kw: mla.mla_splitk_reduce(parts, lses, **kw)
    shares = parts[:, :4].transpose(0, 1).contiguous(), lses[:, :4].t().contiguous()
    out["ranks"] = lambda **kw: mla.mla_dcp_lse_merge_ranks(*shares, **kw)
    rows = dd["pool"].shape[0]
    names = torch.arange(rows, dtype=torch.int32, device="cuda")
    out["gather"] = lambda **kw: mla.mla_debug_gather(dd["pool"], names, **kw)[:1]
    kv = torch.randn(700, 576, generator=g, device="cuda").to(torch.bfloat16)
    qs = torch.randn(700, 16, 192, generator=g, device="cuda").to(torch.bfloat16)
    angles = torch.rand(700, 64, generator=g, device="cuda")
    to = torch.zeros(700, 576, dtype=torch.uint8, device="cuda")
    at = torch.arange(700, dtype=torch.int32, device="cuda")
    out["append"] = lambda **kw: (*mla.mla_cache_append(kv, at, to, at, angles, 1 / 32, q=qs,
                                                        kv_norm_cols=512, **kw), to)
    bytes_ = torch.randint(0, 256, (20000, 576), generator=g, device="cuda", dtype=torch.uint8)
    fork_in = (i32(0, 5000), i32(0, 0), i32(4000, 5000), i32(0, 5000, 10000), 10000,
               torch.arange(6000, 7000, dtype=torch.int32, device="cuda"), i32(0, 1000, 1000))
    five = torch.arange(5000, dtype=torch.int32, device="cuda")
    out["fork"] = lambda **kw: (mla.mla_cache_fork(bytes_, five, *fork_in, **kw), bytes_)
    table = torch.arange(0, 20000, 3, dtype=torch.int32, device="cuda")

    def compact(**kw):
        return mla.mla_cache_compact(bytes_.clone() if not kw else kw.pop("pool"), table, **kw)
    out["compact"] = compact
    return out, bytes_


NAMES = ["prefix", "decode", "dcp", "sparse", "extra", "reduce", "ranks", "gather", "append",
         "fork", "compact"]


@pytest.fixture(scope="module")
def made(_built):
    return calls()


def copied(out):
    return [t.clone() for t in out if t is not None]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("raw", [False, True])
def test_own_memory_on_the_given_stream(made, name, raw):
    fns, bytes_ = made
    want = copied(fns[name]())
    kw = dict(pool=bytes_.clone()) if name == "compact" else {}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):   # what the side stream's pool holds is not zero
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                for n in (1 << 16, 1 << 20, 1 << 24, 1 << 27)]
        del junk
    torch.cuda.synchronize()
    torch.cuda._sleep(PAUSE)        # the current stream is far behind
    behind = torch.cuda.Event()
    behind.record()
    got = fns[name](stream=side.cuda_stream if raw else side, **kw)
    side.synchronize()
    assert not behind.query()       # (else the test shows nothing)
    with torch.cuda.stream(side):
        got = copied(got)
    side.synchronize()
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_does_not_get_it_back_early(made, name):
    fns, bytes_ = made
    want = copied(fns[name]())
    kw = dict(pool=bytes_.clone()) if name == "compact" else {}
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(PAUSE)
    got = fns[name](stream=side, **kw)     # waits behind the pause; its workspace is let go
    for n in (1 << 12, 1 << 16, 1 << 18, 1 << 20, 1 << 22, 1 << 24, 1 << 26):
        for _ in range(4):                  # and would be found here
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.current_stream().synchronize()
    assert not side.query()
    torch.cuda.synchronize()
    for a, b in zip(copied(got), want):
        assert torch.equal(a, b)


def test_default_stream_by_handle_and_other_devices(made, monkeypatch):
    fns, _ = made
    want = copied(fns["prefix"]())
    for handle in (0, 1, torch.cuda.default_stream().cuda_stream):
        got = fns["prefix"](stream=handle)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        fns["prefix"](stream=side)


def test_workspaces_are_zeroed_where_they_have_to_be():
    junk = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    del junk
    s = make(1, 16, 900, [30, 700], seed=74)
    d, plan = to_cuda(s), plan_of(s)
    for ws in (mla.workspace(plan), mla.cache_workspace(), mla.cache_workspace(9000)):
        assert not bool(ws[:mla.MLA_WORKSPACE_HEADER_BYTES].any())
    ws = mla.workspace(plan)
    assert ws.numel() == plan.workspace_bytes
    o, lse = mla.mla_prefix_decode(plan, **d, scale=s.own.scale, kv_scale=s.own.kv_scale,
                                   workspace_t=ws)
    torch.cuda.synchronize()
    compare(o, lse, *oracle.dense_decode(s.joined))
    inp = s.joined
    dplan = mla.mla_decode_plan(2, 1, 16, inp.total_keys, mla.sm_count())
    dd = dense_to_cuda(inp)
    o, lse = mla.mla_decode(dplan, **dd, scale=inp.scale, kv_scale=inp.kv_scale,
                            workspace_t=mla.workspace(dplan))
    torch.cuda.synchronize()
    compare(o, lse, *oracle.dense_decode(inp))
