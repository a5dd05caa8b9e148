"""GPU: the beam and extension calls with ``stream=`` that allocate their own outputs and
workspaces: what a call allocates is zeroed on its stream and belongs to it.  The current
stream may be far behind, or ahead."""
import pytest
import torch

from split_kv_mla_gb300 import mla

pytestmark = pytest.mark.gpu

PAUSE = 100_000_000   # cycles, about 50 ms


def calls():
    g = torch.Generator(device="cuda").manual_seed(80)

    def ints(hi, *shape):
        return torch.randint(0, hi, shape, generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn(48, 30001, generator=g, device="cuda").to(torch.bfloat16)
    s = -9 * torch.rand(8, 6, generator=g, device="cuda")
    state, parents = ints(99999, 40, 5000), ints(40, 40)
    lens, tokens = ints(5000, 40), ints(99, 40)
    sizes = ints(3000, 40)
    ptr = torch.zeros(41, dtype=torch.int32, device="cuda")
    ptr[1:] = sizes.cumsum(0)
    n = int(ptr[-1])
    table = torch.randperm(n + 40, generator=g, device="cuda").int()
    cursor = torch.tensor([0], dtype=torch.int32, device="cuda")
    total = int(sizes[parents.long()].sum()) + 40
    return {
        "select": lambda **kw: mla.mla_beam_select(x, s, 6, end_token=3, **kw),
        "reorder": lambda **kw: mla.mla_beam_reorder(state, parents, lens, tokens, **kw),
        "extend": lambda **kw: mla.mla_cache_extend(table[:n], ptr, sizes, cursor, total, 40, n + 40,
                                                    parents=parents, free_slots=table[n:], **kw)}


@pytest.fixture(scope="module")
def made():
    mla.load()
    return calls()


NAMES = ["select", "reorder", "extend"]


def copied(out):
    return [t.clone() for t in out if t is not None]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("raw", [False, True])
def test_own_memory_on_the_given_stream(made, name, raw):
    want = copied(made[name]())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):   # what the side stream's pool holds is not zero
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                for n in (1 << 16, 1 << 20, 1 << 24)]
        del junk
    torch.cuda.synchronize()
    torch.cuda._sleep(PAUSE)        # the current stream is far behind
    behind = torch.cuda.Event()
    behind.record()
    got = made[name](stream=side.cuda_stream if raw else side)
    side.synchronize()
    assert not behind.query()       # (else the test shows nothing)
    with torch.cuda.stream(side):
        got = copied(got)
    side.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_does_not_get_it_back_early(made, name):
    want = copied(made[name]())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(PAUSE)
    got = made[name](stream=side)     # waits behind the pause; its workspace is let go
    for n in (1 << 9, 1 << 12, 1 << 16, 1 << 18, 1 << 20, 1 << 22):
        for _ in range(4):             # and would be found here
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.current_stream().synchronize()
    assert not side.query()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copied(got), want))


def test_outputs_that_share_an_allocation(made):
    # each of a call's small outputs is a tensor of its own: one outlives the others
    for name in ("select", "extend"):
        want = copied(made[name]())
        kept = []
        for k in range(len(want)):
            kept.append(made[name]()[k])
            for n in (1 << 9, 1 << 11, 1 << 13, 1 << 18):
                torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for got, w in zip(kept, want):
            assert torch.equal(got, w) and got.is_contiguous() and got.data_ptr() % 16 == 0
            got.zero_()               # and can be written to
            assert not bool(got.any())
