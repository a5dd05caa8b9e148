"""Cases, inputs and plain forms of what lies between two steps of a decode loop.

The logits of a step's beams become the next tokens (``mla_beam_select``), the beams'
states follow their parents (``mla_beam_reorder``), and the page tables, lengths, slots
and positions of the next step are built from the requests' lengths
(``mla_cache_extend``).
"""
import math

import torch

own = False

END = 2   # the end token of every case
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one request with four beams: latency of a single user's step
        dict(name="select B1 W4 V32000 bf16", op="select", batch=1, beams=4, vocab=32000, k=4,
             type="bf16", masked=0.0, finished=0, pad=0),
        # a small batch, an odd vocabulary (rows that start on odd elements), twice the beams
        # selected, some beams at their end
        dict(name="select B8 W8 V50001 bf16 K16", op="select", batch=8, beams=8, vocab=50001, k=16,
             type="bf16", masked=0.0, finished=5, pad=0),
        # constrained decoding: nine tenths of the vocabulary masked; rows padded to 100096
        dict(name="select B32 W4 V100003 fp16 masked", op="select", batch=32, beams=4,
             vocab=100003, k=8, type="fp16", masked=0.9, finished=3, pad=93),
        # the largest: 64 requests of eight beams, fp32 logits of a large vocabulary
        dict(name="select B64 W8 V131072 fp32", op="select", batch=64, beams=8, vocab=131072, k=8,
             type="fp32", masked=0.0, finished=0, pad=0),
        # one more token for each request of the headline decode batch
        dict(name="extend F8 S8192", op="extend", requests=8, parents=0, lo=8192, hi=8192, new=1,
             ragged=False, free=True),
        # 64 requests of eight beams that continue their parents' tables
        dict(name="extend F512 S8192 beams", op="extend", requests=512, parents=512, lo=1024,
             hi=8192, new=1, ragged=False, free=True),
        # prefill chunks of up to 2047 tokens behind requests of any length, slots in pool order
        dict(name="extend F61 chunks", op="extend", requests=61, parents=0, lo=0, hi=32768,
             new=2047, ragged=True, free=False),
        # token histories of eight beams
        dict(name="reorder R8 history", op="reorder", rows=8, out=8, cols=2048, type="int32",
             used=700, append=True),
        # rows of odd length, in part in use
        dict(name="reorder R255 C1001 bf16", op="reorder", rows=255, out=255, cols=1001,
             type="bf16", used=900, append=False),
        # states of 512 beams, 256 KB each
        dict(name="reorder R512 C65536 fp32", op="reorder", rows=512, out=512, cols=65536,
             type="fp32", used=0, append=False),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "select", "extend", "reorder"])
    if op == "select":
        batch, beams = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
        vocab = _log(rng, 1000, 262144)
        type_ = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        while batch * beams * vocab > 64 * 8 * 131072:
            batch = max(1, batch // 2)
        return dict(op=op, batch=batch, beams=beams, vocab=vocab,
                    k=rng.choice([beams, beams, 2 * beams, max(1, beams - 1)]), type=type_,
                    masked=rng.choice([0.0, 0.0, 0.5, 0.99]),
                    finished=rng.choice([0, 0, batch * beams // 5]),
                    pad=rng.choice([0, 0, rng.randrange(1, 200)]))
    if op == "extend":
        requests = _log(rng, 1, 1024)
        hi = _log(rng, 16, 32768)
        while requests * hi > 512 * 8192:
            hi //= 2
        ragged = rng.random() < 0.3
        return dict(op=op, requests=requests,
                    parents=rng.choice([0, requests, max(1, requests // 2)]),
                    lo=rng.randrange(0, hi), hi=hi,
                    new=_log(rng, 1, 64) if ragged else rng.choice([1, 1, 2, 4]), ragged=ragged,
                    free=rng.random() < 0.5)
    cols = _log(rng, 16, 65536)
    rows = _log(rng, 1, 512)
    type_ = rng.choice(["int32", "bf16", "fp32"])
    used = rng.choice([0, rng.randrange(1, cols)])
    return dict(op=op, rows=rows, out=rng.choice([rows, rows, max(1, rows // 2)]), cols=cols,
                type=type_, used=used, append=type_ == "int32" and used > 0)


# ---- inputs ---------------------------------------------------------------------------------

def _i32(x):
    return x.to(torch.int32).contiguous()


def _indptr(lens):
    p = torch.zeros(lens.numel() + 1, dtype=torch.int32, device=lens.device)
    p[1:] = torch.cumsum(lens, 0)
    return p


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dev = "cuda"
    s = dict(case)
    op = case["op"]
    if op == "select":
        B, W, V = case["batch"], case["beams"], case["vocab"]
        R = B * W
        x = torch.randn(R, V + case["pad"], generator=g, device=dev).mul_(2.5)
        if case["masked"]:
            off = torch.rand(V, generator=g, device=dev) < case["masked"]
            off[END] = False
            x[:, :V].masked_fill_(off, -math.inf)
        s["logits"] = x.to(TYPES[case["type"]])[:, :V]   # a view of padded rows, if they are padded
        s["scores"] = -5 - 55 * torch.rand(B, W, generator=g, device=dev)
        done = torch.zeros(R, dtype=torch.bool, device=dev)
        done[torch.randperm(R, generator=g, device=dev)[:case["finished"]]] = True
        s["done"] = done.view(B, W)
        if own:
            from split_kv_mla_gb300 import mla
            s["ws"] = mla.beam_workspace(B, W, V)
    elif op == "extend":
        F, NP = case["requests"], case["parents"]
        old = NP or F
        # lengths spread evenly over their range: sizes of the case, not the seed
        parents = None
        if NP:   # the beams of a group of eight have one length, and a parent among themselves
            groups = (old + 7) // 8
            at = torch.arange(old, device=dev) // 8 * 7919 % groups
            lens = case["lo"] + at * (case["hi"] - case["lo"]) // max(1, groups - 1)
            start = torch.arange(F, device=dev) // 8 % groups * 8
            u = torch.rand(F, generator=g, device=dev)
            size = (old - start).clamp(max=8)
            parents = start + torch.minimum((u * size).long(), size - 1)
        else:
            lens = case["lo"] + torch.arange(old, device=dev) * (case["hi"] - case["lo"]) // max(1, old - 1)
            lens = lens[torch.randperm(old, generator=g, device=dev)]
        if case["ragged"]:
            new = (torch.arange(F, device=dev) + 1) * case["new"] // F
            new = new[torch.randperm(F, generator=g, device=dev)]
        else:
            new = torch.full((F,), case["new"], device=dev)
        kept = lens if parents is None else lens[parents]
        T = int(new.sum())
        entries = int(lens.sum())
        rows = entries + T + 4097
        perm = torch.randperm(rows, generator=g, device=dev)
        s["pool_rows"], s["tokens"], s["total"] = rows, T, int(kept.sum()) + T
        s["kv_indices"], s["kv_indptr"], s["seq_lens"] = _i32(perm[:entries]), _indptr(lens), _i32(lens)
        s["new_tokens"] = _i32(new)
        s["parents_t"] = None if parents is None else _i32(parents)
        s["free_slots"] = _i32(perm[entries:]) if case["free"] else None
        s["cursor"] = torch.tensor([1000 if case["free"] else entries], dtype=torch.int32, device=dev)
        if own:
            from split_kv_mla_gb300 import mla
            s["ws"] = mla.cache_workspace()
    else:
        R, F, C = case["rows"], case["out"], case["cols"]
        if case["type"] == "int32":
            s["state"] = torch.randint(0, 50000, (R, C), generator=g, device=dev, dtype=torch.int32)
            s["tokens_t"] = torch.randint(0, 50000, (F,), generator=g, device=dev, dtype=torch.int32)
        else:
            s["state"] = torch.randn(R, C, generator=g, device=dev).to(TYPES[case["type"]])
        group = min(R, 8)
        at = torch.arange(F, device=dev) // group * group
        s["parents_t"] = _i32((at + torch.randint(0, group, (F,), generator=g, device=dev)) % R)
        s["out_t"] = torch.zeros(F, C, dtype=s["state"].dtype, device=dev)
        s["lens"] = None
        if case["used"]:
            spread = torch.arange(R, device=dev) % 8
            s["lens"] = _i32((case["used"] - spread).clamp(min=0))
        if own:
            from split_kv_mla_gb300 import mla
            s["ws"] = mla.cache_workspace()
    return s


# ---- one pass -------------------------------------------------------------------------------

def run(s):
    return {"select": _run_select, "extend": _run_extend, "reorder": _run_reorder}[s["op"]](s)


def _run_select(s):
    B, W, V, K = s["batch"], s["beams"], s["vocab"], s["k"]
    if own:
        from split_kv_mla_gb300 import mla
        return mla.mla_beam_select(s["logits"], s["scores"], K, finished=s["done"], end_token=END,
                                   workspace_t=s["ws"])
    # 64 bits: the scores of different beams lie close to one another
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    x = x.sub_(lse).add_(s["scores"].double().view(-1, 1)).float()
    done = s["done"].view(-1)
    x.masked_fill_(done[:, None], -math.inf)
    x[:, END] = torch.where(done, s["scores"].view(-1), x[:, END])
    # by score, then by the lower index: distinct keys of the two
    bits = x.view(torch.int32).view(B, W * V)
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = bits.long() * (1 << 32) - torch.arange(W * V, device=x.device)
    at = torch.topk(key, K, dim=-1).indices
    scores = x.view(B, W * V).gather(1, at)
    none = scores == -math.inf
    row = torch.arange(B, device=x.device)[:, None] * W
    tokens = torch.where(none, -1, at % V)
    parents = row + torch.where(none, 0, at // V)
    ends = (tokens == END) | none | done[parents]
    return tokens.to(torch.int32), parents.to(torch.int32), scores, ends


def _run_extend(s):
    if own:
        from split_kv_mla_gb300 import mla
        return mla.mla_cache_extend(s["kv_indices"], s["kv_indptr"], s["seq_lens"], s["cursor"],
                                    s["total"], s["tokens"], s["pool_rows"], parents=s["parents_t"],
                                    new_tokens=s["new_tokens"], free_slots=s["free_slots"],
                                    workspace_t=s["ws"])
    new = s["new_tokens"].long()
    F, T, total = new.numel(), s["tokens"], s["total"]
    dev = new.device
    p = torch.arange(F, device=dev) if s["parents_t"] is None else s["parents_t"].long()
    kept = s["seq_lens"].long()[p]
    lens = kept + new
    indptr = torch.zeros(F + 1, dtype=torch.long, device=dev)
    indptr[1:] = torch.cumsum(lens, 0)
    tokptr = torch.zeros(F + 1, dtype=torch.long, device=dev)
    tokptr[1:] = torch.cumsum(new, 0)
    t = torch.arange(T, device=dev)
    ft = torch.searchsorted(tokptr, t, right=True) - 1
    number = s["cursor"].long() + t
    slots = number if s["free_slots"] is None else s["free_slots"].long()[number]
    positions = kept[ft] + t - tokptr[ft]
    i = torch.arange(total, device=dev)
    f = torch.searchsorted(indptr, i, right=True) - 1
    j = i - indptr[f]
    is_old = j < kept[f]
    at = torch.where(is_old, s["kv_indptr"].long()[p[f]] + j, 0)
    table = s["kv_indices"].long()[at] if s["kv_indices"].numel() else at
    fresh = (tokptr[f] + j - kept[f]).clamp(0, max(0, T - 1))
    table = torch.where(is_old, table, slots[fresh]) if T else table
    i32 = torch.int32
    return (table.to(i32), indptr.to(i32), lens.to(i32), slots.to(i32), positions.to(i32),
            tokptr.to(i32), (s["cursor"] + T).to(i32))


def _run_reorder(s):
    if own:
        from split_kv_mla_gb300 import mla
        out, lens = mla.mla_beam_reorder(s["state"], s["parents_t"], lens=s["lens"],
                                         tokens=s["tokens_t"] if s["append"] else None,
                                         out=s["out_t"], workspace_t=s["ws"])
        return (out,) if lens is None else (out, lens)
    p = s["parents_t"].long()
    rows = s["state"][p]
    if s["lens"] is None:
        s["out_t"].copy_(rows)
        return (s["out_t"],)
    lens = s["lens"].long()[p]
    j = torch.arange(s["cols"], device=p.device)
    s["out_t"].copy_(torch.where(j < lens[:, None], rows, s["out_t"]))
    if s["append"]:
        s["out_t"].copy_(torch.where(j == lens[:, None], s["tokens_t"][:, None], s["out_t"]))
        lens = lens + 1
    return s["out_t"], lens.to(torch.int32)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "select":
        R, V = case["batch"] * case["beams"], case["vocab"]
        size = 4 if case["type"] == "fp32" else 2
        live = R - case["finished"]   # a finished beam's logits are not needed
        return dict(bytes=live * V * size + R * 5 + case["batch"] * case["k"] * 13,
                    flops=5.0 * live * V)
    if op == "extend":
        F = case["requests"]
        mean = (case["lo"] + case["hi"]) / 2
        new = F * case["new"] / 2 if case["ragged"] else F * case["new"]
        old = F * mean
        # a parent's entries are read once (a parent has no child in a third of the cases)
        read = old * (0.65 if case["parents"] else 1.0)
        return dict(bytes=(read + old) * 4 + new * (16 if case["free"] else 12) + F * 28, flops=0)
    size = 2 if case["type"] == "bf16" else 4
    cols = case["used"] or case["cols"]
    read = min(case["rows"], case["out"])
    # of eight rows about five are some child's parent: 1 - (7/8)^8
    read = read * 0.65 if read > 1 else read
    return dict(bytes=(read + case["out"]) * cols * size + case["out"] * 12, flops=0)


# ---- the definitions in 64 bits -------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "select":
        B, W, V, K = case["batch"], case["beams"], case["vocab"], case["k"]
        toks, pars, scs, ends = [], [], [], []
        for b in range(B):
            rows = s["logits"][b * W:(b + 1) * W].double()
            score = s["scores"][b].double()[:, None] + torch.log_softmax(rows, -1)
            for w in range(W):
                if bool(s["done"][b, w]):
                    score[w] = -math.inf
                    score[w, END] = s["scores"][b, w].double()
            flat = score.view(-1)
            # scores are numbers of 32 bits: those that round alike are equal
            most = min(flat.numel(), 2 * K + 64)
            edge = torch.topk(flat.float(), most).values[-1]
            cand = (flat.float() >= edge).nonzero()[:, 0] if edge > -math.inf else \
                (flat > -math.inf).nonzero()[:, 0]
            order = torch.sort(flat[cand].float(), descending=True, stable=True).indices[:K]
            at = cand[order]
            n = at.numel()
            tok = torch.full((K,), -1, dtype=torch.int32, device=flat.device)
            par = torch.full((K,), b * W, dtype=torch.int32, device=flat.device)
            sc = torch.full((K,), -math.inf, dtype=torch.float64, device=flat.device)
            end = torch.ones(K, dtype=torch.bool, device=flat.device)
            tok[:n] = (at % V).to(torch.int32)
            par[:n] = (b * W + at // V).to(torch.int32)
            sc[:n] = flat[at]
            end[:n] = (tok[:n] == END) | s["done"][b][at // V]
            toks.append(tok), pars.append(par), scs.append(sc), ends.append(end)
        return torch.stack(toks), torch.stack(pars), torch.stack(scs), torch.stack(ends)
    if op == "extend":
        F = case["requests"]
        n, ip = s["new_tokens"].tolist(), s["kv_indptr"].tolist()
        lens = s["seq_lens"].tolist()
        c = int(s["cursor"])
        dev = s["cursor"].device
        table, ptr, out_lens, slots, pos, tptr = [], [0], [], [], [], [0]
        for f in range(F):
            p = f if s["parents_t"] is None else int(s["parents_t"][f])
            mine = torch.arange(c + tptr[-1], c + tptr[-1] + n[f], device=dev)
            if s["free_slots"] is not None:
                mine = s["free_slots"][mine]
            mine = mine.to(torch.int32)
            table += [s["kv_indices"][ip[p]:ip[p] + lens[p]], mine]
            slots.append(mine)
            pos.append(torch.arange(lens[p], lens[p] + n[f], device=dev, dtype=torch.int32))
            out_lens.append(lens[p] + n[f])
            ptr.append(ptr[-1] + out_lens[-1])
            tptr.append(tptr[-1] + n[f])

        def i32(x):
            return torch.tensor(x, dtype=torch.int32, device=dev)
        return (torch.cat(table), i32(ptr), i32(out_lens), torch.cat(slots), torch.cat(pos),
                i32(tptr), i32([c + tptr[-1]]))
    out = torch.zeros(case["out"], case["cols"], dtype=s["state"].dtype, device="cuda")
    new_lens = []
    for f in range(case["out"]):
        p = int(s["parents_t"][f])
        n = case["cols"] if s["lens"] is None else int(s["lens"][p])
        out[f, :n] = s["state"][p, :n]
        if case["append"]:
            out[f, n] = s["tokens_t"][f]
            n += 1
        new_lens.append(n)
    if s["lens"] is None:
        return (out,)
    return out, torch.tensor(new_lens, dtype=torch.int32, device="cuda")
