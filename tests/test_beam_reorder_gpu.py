"""GPU: beam state reordering.  A copy: everything is exact."""
import pytest
import torch

from split_kv_mla_gb300 import mla

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    mla.load()


def reference(state, parents, lens, tokens, out):
    """(out, out_lens, error bits) of CPU tensors, row by row."""
    out, err, new = out.clone(), 0, []
    cols = state[0].numel() if state.shape[0] else out[0].numel()
    for f, p in enumerate(parents.tolist()):
        if not 0 <= p < state.shape[0]:
            err |= mla.MLA_DEVERR_BAD_TABLE
            new.append(0)
            continue
        n = cols if lens is None else max(0, min(cols, int(lens[p])))
        if lens is not None and n != int(lens[p]):
            err |= mla.MLA_DEVERR_BAD_LENGTH
        out[f].view(-1)[:n] = state[p].reshape(-1)[:n]
        if tokens is not None:
            if n < cols:
                out[f].view(-1)[n] = tokens[f]
                n += 1
            else:
                err |= mla.MLA_DEVERR_BAD_LENGTH
        new.append(n)
    return out, None if lens is None else torch.tensor(new, dtype=torch.int32), err


def bits(t):
    return t.contiguous().view(torch.uint8) if t.numel() else t


def draw(shape, dtype, g):
    n = torch.tensor([], dtype=dtype).element_size()
    for s in shape:
        n *= s
    return torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8).view(dtype).view(shape)


def check(state, parents, lens=None, tokens=None, out=None, **kw):
    ws = mla.cache_workspace()
    c = [None if t is None else t.cpu() for t in (state, parents, lens, tokens)]
    new = torch.zeros((len(c[1]), *state.shape[1:]), dtype=state.dtype) if out is None else out.cpu()
    want, want_lens, err = reference(*c, new)
    got, got_lens = mla.mla_beam_reorder(state, parents, lens, tokens, out, workspace_t=ws, **kw)
    torch.cuda.synchronize()
    assert mla.mla_read_device_error(ws) == err
    assert out is None or got is out
    assert torch.equal(bits(got.cpu()), bits(want))
    assert (got_lens is None) == (lens is None)
    assert lens is None or torch.equal(got_lens.cpu(), want_lens)


@pytest.mark.parametrize("dtype", [torch.uint8, torch.bfloat16, torch.int32, torch.float32,
                                   torch.int64])
@pytest.mark.parametrize("R,F,cols", [(1, 1, 1), (3, 5, 7), (8, 8, 16), (5, 9, 1001), (2, 3, 4096),
                                      (40, 17, 4099), (3, 1, 20000), (700, 900, 33)])
def test_whole_rows(dtype, R, F, cols):
    g = torch.Generator().manual_seed(cols)
    state = draw((R, cols), dtype, g).cuda()
    parents = torch.randint(0, R, (F,), generator=g).int().cuda()
    check(state, parents)
    check(state, parents, out=draw((F, cols), dtype, g).cuda())


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float16, torch.int32, torch.float64])
@pytest.mark.parametrize("cols", [1, 15, 16, 17, 1000, 1001, 8200])
def test_lengths_leave_the_rest(dtype, cols):
    g = torch.Generator().manual_seed(cols)
    R, F = 13, 21
    state = draw((R, cols), dtype, g).cuda()
    parents = torch.randint(0, R, (F,), generator=g).int().cuda()
    lens = torch.randint(0, cols + 1, (R,), generator=g).int()
    lens[0], lens[1], lens[2] = 0, cols, 1
    check(state, parents, lens.cuda(), out=draw((F, cols), dtype, g).cuda())
    check(state, parents, lens.cuda())
    if dtype == torch.int32:
        tokens = torch.randint(0, 99999, (F,), generator=g).int().cuda()
        check(state, parents, (lens - 1).clamp(min=0).cuda(), tokens,
              out=draw((F, cols), dtype, g).cuda())
        check(state, parents, lens.cuda(), tokens)    # a row without room


@pytest.mark.parametrize("dtype", [torch.uint8, torch.bfloat16, torch.int32])
@pytest.mark.parametrize("shift,pad", [(0, 16), (1, 0), (2, 3), (4, 4), (8, 24), (16, 7)])
def test_strides_and_alignments(dtype, shift, pad):
    g = torch.Generator().manual_seed(shift)
    R, F, cols = 6, 7, 500

    def view(rows, shift, pad, shape=(500,)):
        n = rows * (cols + pad) + shift
        return draw((n,), dtype, g).cuda()[shift:].as_strided((rows, *shape), (cols + pad, *(
            (1,) if len(shape) == 1 else (shape[1], 1))))
    parents = torch.randint(0, R, (F,), generator=g).int().cuda()
    check(view(R, shift, pad), parents, out=view(F, 0, 0))
    check(view(R, 0, pad), parents, out=view(F, shift, pad + 1))
    check(view(R, shift, pad, (5, 100)), parents, out=view(F, shift, pad, (5, 100)))
    lens = torch.randint(0, cols + 1, (R,), generator=g).int().cuda()
    out = view(F, shift, pad)
    whole = out.as_strided((F, cols + pad), (cols + pad, 1))[:-1]
    before = whole.clone()
    check(view(R, 1, pad), parents, lens, out=out)
    assert torch.equal(bits(whole[:, cols:]), bits(before[:, cols:]))    # between the rows
    # rows of state and out in turn in one buffer
    both = draw((8, 2, cols), dtype, g).cuda()
    check(both[:, 0], torch.arange(7, -1, -1).int().cuda(), out=both[:, 1])


def test_bad_parents_and_lengths():
    g = torch.Generator().manual_seed(3)
    state = draw((5, 70), torch.int32, g).cuda()
    out = draw((6, 70), torch.int32, g).cuda()
    parents = torch.tensor([0, -1, 4, 5, 1 << 30, 2]).int().cuda()
    check(state, parents, out=out.clone())
    tokens = torch.arange(6).int().cuda()
    check(state, parents, torch.tensor([3, 1, 70, 1, 69]).int().cuda(), tokens, out=out.clone())
    check(state, parents, torch.tensor([-3, 71, 1 << 30, 5, -1 << 31]).int().cuda(), tokens,
          out=out.clone())
    check(state[:0], parents, out=out.clone())
    check(state, parents[:0])
    check(state[:, :0], parents)


def test_rows_behind_four_gigabytes():
    # 2^18 columns of 8 bytes, 2049 rows: the last at 2^32 bytes
    state = torch.zeros(2049, 1 << 18, dtype=torch.int64, device="cuda")
    state[2048] = torch.arange(1 << 18, device="cuda")
    state[2047] = -7
    out, _ = mla.mla_beam_reorder(state, torch.tensor([2048, 2047, 2048]).int().cuda())
    assert torch.equal(out[0], state[2048]) and bool((out[1] == -7).all())
    assert torch.equal(out[2], out[0])
    out, _ = mla.mla_beam_reorder(out, (torch.arange(2049) % 3).int().cuda(), out=state)
    assert torch.equal(state[2048], torch.full_like(state[0], 0) + out[2])
    del state, out
    torch.cuda.empty_cache()


def test_captured_in_place_refused_and_streams():
    g = torch.Generator().manual_seed(5)
    a, b = draw((8, 300), torch.int32, g).cuda(), torch.zeros(8, 300, dtype=torch.int32).cuda()
    lens = torch.full((8,), 10, dtype=torch.int32, device="cuda")
    lens2 = torch.zeros_like(lens)
    parents, tokens = torch.zeros(8).int().cuda(), torch.zeros(8).int().cuda()
    ws = mla.cache_workspace()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):   # two steps, there and back
        mla.mla_beam_reorder(a, parents, lens, tokens, b, lens2, workspace_t=ws)
        mla.mla_beam_reorder(b, parents, lens2, tokens, a, lens, workspace_t=ws)
    ca, cb, cl = a.cpu(), b.cpu(), lens.cpu()
    for step in range(4):
        parents.copy_(torch.randint(0, 8, (8,), generator=g))
        tokens.copy_(torch.randint(0, 999, (8,), generator=g))
        graph.replay()
        cb, cl, _ = reference(ca, parents.cpu(), cl, tokens.cpu(), cb)
        ca, cl, _ = reference(cb, parents.cpu(), cl, tokens.cpu(), ca)
        torch.cuda.synchronize()
        assert torch.equal(a.cpu(), ca) and torch.equal(b.cpu(), cb) and torch.equal(lens.cpu(), cl)
    assert mla.mla_read_device_error(ws) == 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, _ = mla.mla_beam_reorder(a, parents, stream=side)
    side.synchronize()
    assert torch.equal(got, a[parents.long()])
    kw = dict(workspace_t=ws)
    for bad in (dict(out=a), dict(out=a.view(-1)[1200:].view(4, 300)), dict(tokens=tokens),
                dict(out_lens=lens), dict(lens=lens, out_lens=lens), dict(lens=lens[:7]),
                dict(lens=lens, tokens=tokens[:7]), dict(out=b.float()), dict(out=b[:7]),
                dict(out=b.view(8, 30, 10)[:, :, :5]), dict(lens=lens.long())):
        with pytest.raises((ValueError, mla.MlaError)):
            mla.mla_beam_reorder(a, parents, **bad, **kw)
    for state, par in ((a.t(), parents), (a.cpu(), parents), (a, parents.long()), (a[0, 0], parents),
                       (a.to(torch.complex128), parents)):
        with pytest.raises((ValueError, mla.MlaError)):
            mla.mla_beam_reorder(state, par, **kw)
