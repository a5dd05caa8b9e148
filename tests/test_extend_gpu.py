"""GPU: cache extension against a plain Python build of the tables.  Whole numbers: exact."""
import pytest
import torch

from split_kv_mla_gb300 import mla

pytestmark = pytest.mark.gpu

BAD_SLOT, BAD_LENGTH = mla.MLA_DEVERR_BAD_SLOT, mla.MLA_DEVERR_BAD_LENGTH
BAD_TABLE, NO_SLOT = mla.MLA_DEVERR_BAD_TABLE, mla.MLA_DEVERR_NO_SLOT
MARK = -77   # what outputs hold before the call


@pytest.fixture(scope="module", autouse=True)
def _built():
    mla.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def reference(c):
    """Outputs and error bits of a case (lists), request by request."""
    ip, idx, lens = c["kv_indptr"], c["kv_indices"], c["seq_lens"]
    F = len(c["parents"]) if c.get("parents") is not None else \
        len(c["new_tokens"]) if c.get("new_tokens") is not None else len(lens)
    total, T, cur = c["total"], c["num_tokens"], c["cursor"]
    prefix = c.get("prefix_len") or 0
    table, slots, positions = [MARK] * total, [-1] * T, [0] * T
    indptr, tokptr, out_lens, err, t, e = [0], [0], [], 0, 0, 0
    for f in range(F):
        p = f if c.get("parents") is None else c["parents"][f]
        n = 1 if c.get("new_tokens") is None else c["new_tokens"][f]
        keep = 0
        if not 0 <= p < len(lens) or not 0 <= ip[p] <= ip[p + 1] <= len(idx):
            err |= BAD_TABLE
            p = None
        else:
            keep = max(0, min(lens[p], ip[p + 1] - ip[p]))
            err |= BAD_LENGTH if keep != lens[p] else 0
        if n < 0:
            n, err = 0, err | BAD_LENGTH
        if n > T - t:
            n, err = T - t, err | BAD_TABLE
        length = keep + n
        if length > total - e:
            length, err = total - e, err | BAD_TABLE
        for j in range(min(keep, length)):
            table[e + j] = idx[ip[p] + j]
        for i in range(n):
            positions[t + i] = keep + i + prefix
            if keep + i >= length:
                continue
            number = cur + t + i
            free = c.get("free_slots")
            if not 0 <= number < (c["pool_rows"] if free is None else len(free)):
                slot, err = -1, err | NO_SLOT
            else:
                slot = number if free is None else free[number]
                if not 0 <= slot < c["pool_rows"]:
                    slot, err = -1, err | BAD_SLOT
            slots[t + i] = table[e + keep + i] = slot
        t, e = t + n, e + length
        indptr.append(e)
        tokptr.append(t)
        out_lens.append(length)
    after = (cur + t + (1 << 31)) % (1 << 32) - (1 << 31)
    return (table, indptr, out_lens, slots, positions, tokptr, [after]), err


NAMES = ("kv_indices", "kv_indptr", "seq_lens", "parents", "new_tokens", "free_slots")


def on_gpu(c):
    d = {k: i32(c[k]).cuda() for k in NAMES if c.get(k) is not None}
    d["cursor"] = i32([c["cursor"]]).cuda()
    if c.get("prefix_len") is not None:
        d["prefix_len"] = i32([c["prefix_len"]]).cuda()
    return dict(d, total=c["total"], num_tokens=c["num_tokens"], pool_rows=c["pool_rows"])


def check(c, inplace=False):
    d = on_gpu(c)
    want, err = reference(c)
    ws = mla.cache_workspace()
    full = [torch.full((len(w),), MARK, dtype=torch.int32, device="cuda") for w in want]
    names = ("table", "indptr", "lens", "slots", "positions", "token_indptr", "new_cursor")
    out = dict(zip(names, full))
    if inplace:
        out["new_cursor"] = d["cursor"]
    got = mla.mla_cache_extend(**d, **out, workspace_t=ws)
    torch.cuda.synchronize()
    assert mla.mla_read_device_error(ws) == err
    for name, g, w in zip(names, got, want):
        assert g is out[name]
        assert g.tolist() == w, name
    return got


def make(lens, seed=0, parents=None, new=None, free=False, spare=0, prefix=None, room=0):
    """Tables of the lengths (with `spare` entries behind each) in a shuffled pool."""
    g = torch.Generator().manual_seed(seed)
    spans = [n + spare for n in lens]
    F = len(parents) if parents is not None else len(new) if new is not None else len(lens)
    counts = [1] * F if new is None else new
    T = sum(max(0, n) for n in counts)
    rows = sum(spans) + T + 40
    perm = torch.randperm(rows, generator=g).tolist()
    indptr = [0]
    for n in spans:
        indptr.append(indptr[-1] + n)
    kept = [lens[p] for p in (range(F) if parents is None else parents)]
    return dict(kv_indices=perm[:sum(spans)], kv_indptr=indptr, seq_lens=list(lens), parents=parents,
                new_tokens=new, free_slots=perm[sum(spans):] if free else None,
                cursor=7 if free else sum(spans), pool_rows=rows, total=sum(kept) + T + room,
                num_tokens=T + room, prefix_len=prefix)


@pytest.mark.parametrize("free", [False, True])
@pytest.mark.parametrize("lens", [[0], [1], [5], [0, 0, 0], [1, 0, 3], [255, 256, 257], [1000],
                                  list(range(70)), [4096, 1, 5000, 0, 31]])
def test_one_more_token(lens, free):
    check(make(lens, free=free))
    check(make(lens, free=free, spare=3), inplace=True)
    check(make(lens, free=free, new=[1] * len(lens), prefix=1234))


@pytest.mark.parametrize("seed", range(6))
def test_beams_and_ragged_counts(seed):
    g = torch.Generator().manual_seed(seed)

    def ints(lo, hi, n):
        return torch.randint(lo, hi, (n,), generator=g).tolist()
    R, F = ints(1, 60, 1)[0], ints(1, 200, 1)[0]
    lens = ints(0, [3, 40, 700, 3000, 130, 1][seed], R)
    parents = ints(0, R, F)
    check(make(lens, seed, parents))
    check(make(lens, seed, parents, new=ints(0, 5, F), free=True, spare=2, room=9))
    check(make(lens, seed, parents, new=ints(0, 900, F), prefix=3))
    check(make(lens, seed, None, new=ints(0, 300, R), free=True), inplace=True)
    check(make(lens, seed, None, new=ints(0, 3, max(1, R // 2)), free=True))


@pytest.mark.parametrize("F", [1023, 1024, 1025, 2048, 2049, 4100, 9000])
def test_many_requests(F):
    g = torch.Generator().manual_seed(F)
    lens = torch.randint(0, 20, (F,), generator=g).tolist()
    check(make(lens, F, new=torch.randint(0, 3, (F,), generator=g).tolist(), free=True, room=5))
    parents = torch.randint(0, F, (F,), generator=g).tolist()
    check(make(lens, F, parents), inplace=True)


def test_no_requests_and_no_tokens():
    check(make([], new=[], room=6))
    check(make([4, 9], parents=[], room=3))
    check(make([4, 9], new=[0, 0]))
    check(make([4, 9], new=[0, 0], room=4))
    check(make([0, 0], new=[0, 0]))


def test_lengths_drop_the_last_positions():
    c = make([9, 30, 4], spare=5, free=True)      # four drafts each, some accepted
    c["seq_lens"] = [12, 35, 4]
    c["total"] = 12 + 35 + 4 + 3
    check(c)


@pytest.mark.parametrize("lens", [[10, 20, 30], [3] * 3000])
def test_what_the_device_finds_wrong(lens):
    base = make(lens, new=[2] * len(lens), free=True, room=5)
    n = len(lens)

    def case(**kw):
        check(dict(base, **kw))
    case(seq_lens=[lens[0] + 1, -4] + lens[2:])
    case(new_tokens=[-1, 2] + [2] * (n - 2))
    case(parents=[0, -1] + [n, 1 << 30] + [1] * (n - 4) if n > 3 else [0, -1, 3])
    case(kv_indptr=[0, lens[0]] + [-5] + base["kv_indptr"][3:])
    case(kv_indptr=base["kv_indptr"][:-1] + [sum(lens) + 1])
    case(kv_indptr=base["kv_indptr"][:-1] + [0])
    case(cursor=len(base["free_slots"]) - 3)       # three slots are left
    case(cursor=-2)
    case(cursor=len(base["free_slots"]) + 100)
    case(free_slots=base["free_slots"][:9] + [-1, base["pool_rows"]] + base["free_slots"][11:])
    case(pool_rows=base["pool_rows"] // 2)
    case(total=sum(lens) // 2)                     # no room
    case(total=0)
    case(num_tokens=3)
    case(num_tokens=0)
    case(num_tokens=n, total=sum(lens))
    case(free_slots=None, cursor=base["pool_rows"] - 4)
    case(free_slots=None, cursor=(1 << 31) - 2, num_tokens=2)


def test_prefix_and_large_positions():
    c = make([5, 6], prefix=1 << 30)
    check(c)


def test_a_large_table():
    g = torch.Generator(device="cuda").manual_seed(1)
    F, L = 900, 9001
    lens = torch.randint(0, L, (F,), generator=g, device="cuda")
    parents = torch.randint(0, F, (F,), generator=g, device="cuda")
    n = int(lens.sum())
    perm = torch.randperm(n + 70000, generator=g, device="cuda").int()
    new = torch.randint(0, 100, (F,), generator=g, device="cuda")
    ptr = torch.zeros(F + 1, dtype=torch.int32, device="cuda")
    ptr[1:] = lens.cumsum(0)
    T, total = int(new.sum()), int(lens[parents].sum() + new.sum())
    cursor = torch.zeros(1, dtype=torch.int32, device="cuda")
    table, indptr, out_lens, slots, positions, tokptr, after = mla.mla_cache_extend(
        perm[:n], ptr, lens.int(), cursor, total, T, n + 70000, parents=parents.int(),
        new_tokens=new.int(), free_slots=perm[n:])
    assert int(after) == T and int(indptr[-1]) == total and int(tokptr[-1]) == T
    assert torch.equal(slots, perm[n:n + T])
    want = []
    for f in range(F):
        p, a = int(parents[f]), int(tokptr[f])
        m = int(lens[p])
        want += [perm[int(ptr[p]):int(ptr[p]) + m], slots[a:a + int(new[f])]]
        assert int(out_lens[f]) == m + int(new[f])
    assert torch.equal(table, torch.cat(want))
    where = torch.repeat_interleave(torch.arange(F, device="cuda"), new)
    at = torch.arange(T, device="cuda") - tokptr[:-1].long()[where]
    assert torch.equal(positions.long(), lens[parents[where]] + at)


def test_captured_steps_and_compaction():
    # a graph of two steps, there and back, with the cursor in place; the lengths that it
    # finds are the device's
    c = dict(make([9, 30, 4], room=300), kv_indices=list(range(43)))
    d = on_gpu(dict(c, pool_rows=2000))
    cap = 43 + 300
    a = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (cap, 4, 3)]
    b = [t.clone() for t in a]
    for t, v in zip(a, (c["kv_indices"], c["kv_indptr"], c["seq_lens"])):
        t[:len(v)] = i32(v).cuda()
    cursor, ws = d["cursor"], mla.cache_workspace()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, y in ((a, b), (b, a)):
            mla.mla_cache_extend(*x, cursor, cap, 3, 2000, table=y[0], indptr=y[1], lens=y[2],
                                 new_cursor=cursor, workspace_t=ws)
    state = dict(c, total=cap, num_tokens=3, pool_rows=2000)
    for step in range(10):
        graph.replay()
        for _ in range(2):
            want, err = reference(state)
            assert err == 0
            state.update(kv_indices=want[0], kv_indptr=want[1], seq_lens=want[2], cursor=want[6][0])
        torch.cuda.synchronize()
        n = want[1][-1]
        assert a[0][:n].tolist() == want[0][:n]
        assert a[1].tolist() == want[1] and a[2].tolist() == want[2]
        assert int(cursor) == want[6][0]
    assert mla.mla_read_device_error(ws) == 0
    # what compaction calls live is the next cursor
    pool = torch.zeros(2000, 576, dtype=torch.uint8, device="cuda")
    table, live = mla.mla_cache_compact(pool, a[0][:n].clone())
    out = mla.mla_cache_extend(table, a[1], a[2], live, n + 3, 3, 2000, new_cursor=live)
    used = out[0].tolist()
    assert sorted(used) == list(range(n + 3)) and int(live) == n + 3


def test_refusals_and_streams():
    d = on_gpu(make([5, 6, 7], new=[1, 2, 3], free=True))
    ws = mla.cache_workspace()
    want = mla.mla_cache_extend(**d, workspace_t=ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mla.mla_cache_extend(**d, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    for bad in (dict(table=d["kv_indices"]), dict(lens=d["seq_lens"]), dict(indptr=d["kv_indptr"]),
                dict(total=-1), dict(num_tokens=-1), dict(pool_rows=-1), dict(pool_rows=1 << 31),
                dict(table=torch.zeros(5, dtype=torch.int32, device="cuda")),
                dict(slots=torch.zeros(6, device="cuda")), dict(new_tokens=d["new_tokens"][:2],
                                                               parents=d["seq_lens"]),
                dict(new_tokens=torch.ones(4, dtype=torch.int32, device="cuda")),
                dict(seq_lens=d["seq_lens"][:2]), dict(cursor=d["seq_lens"]),
                dict(prefix_len=d["seq_lens"]), dict(kv_indices=d["kv_indices"].cpu()),
                dict(kv_indptr=d["kv_indptr"].long())):
        with pytest.raises((ValueError, mla.MlaError)):
            mla.mla_cache_extend(**dict(d, **bad), workspace_t=ws)
