"""Cases, inputs and plain forms of the cache and shared-prefix operators.

A shared prefix's life in the paged fp8 cache: a prompt's rows are normed,
rotated, quantised and appended (``mla_cache_append``), forked to several
requests (``mla_cache_fork``), decoded with the prefix computed once for the
whole batch (``mla_prefix_decode``), and the slots that nobody names any more
are compacted away (``mla_cache_compact``).
"""
import math

import torch

own = False

D_ROPE = 64
KV_SCALE = 1.0 / 32.0
EPS = 1e-6


def listed():
    return [
        # a few chat requests on a short system prompt: latency of one small step
        dict(name="prefix B4 H16 P1024", op="prefix", batch=4, q_len=1, heads=16, prefix=1024,
             lo=1, hi=64),
        # a batch of 64 on one document of the repository's headline length
        dict(name="prefix B64 H16 P8192", op="prefix", batch=64, q_len=1, heads=16, prefix=8192,
             lo=16, hi=512),
        # speculative verify of 4 draft tokens, odd prefix, requests that have just begun
        dict(name="prefix B8 H16 q4 P32001", op="prefix", batch=8, q_len=4, heads=16, prefix=32001,
             lo=1, hi=300),
        # the largest: 128 heads, 64 requests, a 32k prefix
        dict(name="prefix B64 H128 P32768", op="prefix", batch=64, q_len=1, heads=128,
             prefix=32768, lo=1, hi=1024),
        # one decode step's append for 8 requests of 16 heads
        dict(name="append T8 H16", op="append", tokens=8, heads=16, width=576, q_cols=64,
             q_norm=False, half=False, pool=65536, holes=0),
        # a prefill chunk of 8192 tokens, 128 heads (128 non-rotated + 64 rotated columns)
        dict(name="append T8192 H128", op="append", tokens=8192, heads=128, width=576, q_cols=192,
             q_norm=False, half=False, pool=65536, holes=0),
        # the 448+64 row form, queries normed for each head, an odd chunk with padded tokens
        dict(name="append T4093 H64 w512", op="append", tokens=4093, heads=64, width=512,
             q_cols=512, q_norm=True, half=True, pool=65536, holes=37),
        # a request forked into two that copy its last unshared rows
        dict(name="fork F2 S700", op="fork", children=2, parents=1, length=700, keep=640,
             width=576, pool=65536),
        # 64 samples of 8 prompts that share half of the prompt and own the rest
        dict(name="fork F64 S8192", op="fork", children=64, parents=8, length=8192, keep=4096,
             width=576, pool=524288),
        # a small cache after some requests have ended
        dict(name="compact N8192", op="compact", pool=8192, live=3000, requests=8, width=576),
        # the sparse row form, half full
        dict(name="compact N131072 w512", op="compact", pool=131072, live=65000, requests=32,
             width=512),
        # a large cache, four tenths live
        dict(name="compact N1048576", op="compact", pool=1048576, live=419431, requests=64,
             width=576),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "append", "fork", "compact"])
    if op == "prefix":
        heads = rng.choice([1, 8, 16, 16, 64, 128])
        q_len = rng.choice([1, 1, 1, 2, 4])
        batch = _log(rng, 1, 64)
        prefix = _log(rng, 64, 32768)
        while batch * q_len * heads * prefix > 64 * 128 * 32768:
            prefix //= 2
        lo = rng.choice([0, 1, 16])
        return dict(op=op, batch=batch, q_len=q_len, heads=heads, prefix=prefix, lo=lo,
                    hi=lo + _log(rng, 1, 1024))
    if op == "append":
        width = rng.choice([576, 512])
        heads = rng.choice([1, 8, 16, 64, 128])
        tokens = _log(rng, 1, 8192)
        q_cols = rng.choice([64, 192]) if width == 576 else 512
        if q_cols == 512:
            while tokens * heads > 4096 * 64:
                tokens //= 2
        return dict(op=op, tokens=tokens, heads=heads, width=width, q_cols=q_cols,
                    q_norm=rng.random() < 0.5, half=rng.random() < 0.5, pool=65536,
                    holes=rng.choice([0, 0, tokens // 7]))
    if op == "fork":
        length = _log(rng, 16, 8192)
        return dict(op=op, children=_log(rng, 1, 64), parents=rng.choice([1, 2, 8]),
                    length=length, keep=rng.randrange(length // 2, length + 1),
                    width=rng.choice([576, 512]), pool=524288)
    pool = _log(rng, 256, 1 << 20)
    return dict(op=op, pool=pool, live=rng.randrange(1, pool), requests=_log(rng, 1, 64),
                width=rng.choice([576, 512]))


# ---- inputs ---------------------------------------------------------------------------------

def _pool(rows, width, g):
    """fp8 bytes [rows, width] of N(0, 1) / KV_SCALE."""
    x = torch.randn(rows, width, generator=g, device="cuda") / KV_SCALE
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _i32(x):
    return x.to(torch.int32).contiguous()


def _indptr(lens):
    p = torch.zeros(lens.numel() + 1, dtype=torch.int32, device="cuda")
    p[1:] = torch.cumsum(lens, 0)
    return p


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dev = "cuda"
    s = dict(case)
    op = case["op"]
    if op == "prefix":
        B, Q, H, P = case["batch"], case["q_len"], case["heads"], case["prefix"]
        lens = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=g, device=dev)
        total, s["most"] = int(lens.sum()), int(lens.max())
        rows = P + total + 999
        s["pool_t"] = _pool(rows, 576, g)
        perm = torch.randperm(rows, generator=g, device=dev)
        s["prefix_indices"] = _i32(perm[:P])
        s["kv_indices"] = _i32(perm[P:P + total])
        s["seq_lens"], s["kv_indptr"] = _i32(lens), _indptr(lens)
        s["prefix_len"] = torch.tensor([P], dtype=torch.int32, device=dev)
        s["q_lat"] = torch.randn(B * Q, H, 512, generator=g, device=dev).to(torch.bfloat16)
        s["q_pe"] = torch.randn(B * Q, H, D_ROPE, generator=g, device=dev).to(torch.bfloat16)
        s["scale"] = 576 ** -0.5
        if own:
            from split_kv_mla_gb300 import mla
            s["plan"] = mla.mla_prefix_decode_plan(B, Q, H, P, total, mla.sm_count())
            s["ws"] = mla.workspace(s["plan"])
    elif op == "append":
        T, H, W, D = case["tokens"], case["heads"], case["width"], case["q_cols"]
        s["kv"] = torch.randn(T, W, generator=g, device=dev).to(torch.bfloat16)
        s["kv_weight"] = (1 + 0.1 * torch.randn(W - 64 if W == 576 else W, generator=g,
                                                device=dev)).to(torch.bfloat16)
        s["q"] = torch.randn(T, H, D, generator=g, device=dev).to(torch.bfloat16)
        s["q_weight"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16)
        s["positions"] = torch.randint(0, 131072, (T,), generator=g, device=dev,
                                       dtype=torch.int32)
        inv = 10000.0 ** (-torch.arange(32, device=dev, dtype=torch.float64) / 32)
        ang = torch.arange(131072, device=dev, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        slots = torch.randperm(case["pool"], generator=g, device=dev)[:T]
        if case["holes"]:
            slots[torch.randperm(T, generator=g, device=dev)[:case["holes"]]] = -1
        s["slots"] = _i32(slots)
        s["pool_t"] = _pool(case["pool"], W, g)
        if own:
            from split_kv_mla_gb300 import mla
            s["ws"] = mla.cache_workspace()
    elif op == "fork":
        F, NP, L, K = case["children"], case["parents"], case["length"], case["keep"]
        # lengths a little apart, and children dealt out in turn: sizes of the case, not the seed
        lens = L - torch.arange(NP, device=dev) * 5 % 8
        parent = torch.arange(F, device=dev) % NP
        total = int(lens.sum())
        keep = torch.minimum(torch.full((F,), K, device=dev), lens[parent])
        fresh = lens[parent] - keep
        nfresh = int(fresh.sum())
        perm = torch.randperm(case["pool"], generator=g, device=dev)
        s["pool_t"] = _pool(case["pool"], case["width"], g)
        s["kv_indices"], s["kv_indptr"] = _i32(perm[:total]), _indptr(lens)
        s["parents_t"], s["keep_t"] = _i32(parent), _i32(keep)
        s["child_indptr"], s["total"] = _indptr(lens[parent]), int(lens[parent].sum())
        s["fresh"], s["fresh_indptr"] = _i32(perm[total:total + nfresh]), _indptr(fresh)
        if own:
            from split_kv_mla_gb300 import mla
            s["ws"] = mla.cache_workspace()
    else:
        N, R = case["pool"], case["requests"]
        live = torch.randperm(N, generator=g, device=dev)[:case["live"]]
        # each request shares a first piece with the others: slots named more than once
        share = live[:max(1, case["live"] // 8)]
        s["kv_indices"] = _i32(torch.cat([live] + [share] * min(R - 1, 7) +
                                         [torch.full((5,), -1, device=dev)]))
        s["pool_t"] = _pool(N, case["width"], g)
        if own:
            from split_kv_mla_gb300 import mla
            s["ws"] = mla.cache_workspace(N)
    return s


# ---- one pass -------------------------------------------------------------------------------

def run(s):
    return {"prefix": _run_prefix, "append": _run_append, "fork": _run_fork,
            "compact": _run_compact}[s["op"]](s)


def _run_prefix(s):
    if own:
        from split_kv_mla_gb300 import mla
        return mla.mla_prefix_decode(s["plan"], s["q_lat"], s["q_pe"], s["pool_t"],
                                     s["prefix_indices"], s["seq_lens"], s["kv_indices"],
                                     s["kv_indptr"], s["scale"], KV_SCALE,
                                     prefix_len=s["prefix_len"], workspace_t=s["ws"])
    B, Q, H, P, M = s["batch"], s["q_len"], s["heads"], s["prefix"], s["most"]
    q = torch.cat([s["q_lat"], s["q_pe"]], -1).float().view(B, Q * H, 576)
    lens = s["seq_lens"].long()
    kp = s["pool_t"][s["prefix_indices"].long()].view(torch.float8_e4m3fn).float() * KV_SCALE
    j = torch.arange(M, device=q.device)
    at = (s["kv_indptr"][:-1].long()[:, None] + j).clamp(max=max(0, s["kv_indices"].numel() - 1))
    slots = s["kv_indices"].long()[at] if s["kv_indices"].numel() else at
    ks = s["pool_t"][slots].view(torch.float8_e4m3fn).float() * KV_SCALE
    # draft row t sees positions up to P + len - q_len + t
    last = (P + lens[:, None] - Q + torch.arange(Q, device=q.device)).repeat_interleave(H, 1)
    sp = (q.view(-1, 576) @ kp.T).view(B, Q * H, P) * s["scale"]
    sp.masked_fill_(torch.arange(P, device=q.device) > last[..., None], -math.inf)
    ss = torch.bmm(q, ks.transpose(1, 2)) * s["scale"]
    ss.masked_fill_((P + j > last[..., None]) | (j >= lens[:, None, None]), -math.inf)
    m = sp.amax(-1) if M == 0 else torch.maximum(sp.amax(-1), ss.amax(-1))
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)[..., None]
    ep, es = torch.exp(sp - m0), torch.exp(ss - m0)
    l = ep.sum(-1) + es.sum(-1)
    o = (ep.view(-1, P) @ kp[:, :512]).view(B, Q * H, 512) + torch.bmm(es, ks[..., :512])
    o = torch.where(l[..., None] > 0, o / l[..., None], torch.zeros_like(o))
    lse = (m0[..., 0] + torch.log(l)) / math.log(2.0)
    return o.to(torch.bfloat16).view(B * Q, H, 512), lse.view(B * Q, H)


def _rotate(x, cos, sin, half):
    """x [..., 64] with pairs (i, i + 32) or (2 i, 2 i + 1) turned by the angles."""
    a, b = (x[..., :32], x[..., 32:]) if half else (x[..., 0::2], x[..., 1::2])
    y, z = a * cos - b * sin, b * cos + a * sin
    return torch.cat([y, z], -1) if half else torch.stack([y, z], -1).flatten(-2)


def _run_append(s):
    W, D = s["width"], s["q_cols"]
    dv = W - 64
    if own:
        from split_kv_mla_gb300 import mla
        q_nope, q_pe = mla.mla_cache_append(
            s["kv"], s["slots"], s["pool_t"], s["positions"], s["cos_sin"], KV_SCALE, q=s["q"],
            kv_weight=s["kv_weight"], kv_norm_cols=dv if W == 576 else W,
            q_weight=s["q_weight"] if s["q_norm"] else None, q_norm=s["q_norm"], eps=EPS,
            half_split=s["half"], workspace_t=s["ws"])
    else:
        n = dv if W == 576 else W
        kv = s["kv"].float()
        r = torch.rsqrt(kv[:, :n].square().mean(-1, keepdim=True) + EPS)
        kv[:, :n] = kv[:, :n] * r * s["kv_weight"].float()
        cs = s["cos_sin"][s["positions"].long()]
        cos, sin = cs[:, :32], cs[:, 32:]
        kv[:, dv:] = _rotate(kv[:, dv:], cos, sin, s["half"])
        row = (kv / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        on = s["slots"] >= 0
        s["pool_t"][s["slots"][on].long()] = row[on]
        q = s["q"].float()
        if s["q_norm"]:
            r = torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS)
            q = q * r * s["q_weight"].float()
        q_pe = _rotate(q[..., -64:], cos[:, None], sin[:, None], s["half"]).to(torch.bfloat16)
        q_nope = q[..., :-64].to(torch.bfloat16) if D > 64 else None
    pool = s["pool_t"].view(torch.float8_e4m3fn)
    return (pool, q_pe) if q_nope is None else (pool, q_pe, q_nope)


def _run_fork(s):
    if own:
        from split_kv_mla_gb300 import mla
        table = mla.mla_cache_fork(s["pool_t"], s["kv_indices"], s["kv_indptr"], s["parents_t"],
                                   s["keep_t"], s["child_indptr"], s["total"], s["fresh"],
                                   s["fresh_indptr"], workspace_t=s["ws"])
    else:
        i = torch.arange(s["total"], device="cuda")
        f = torch.searchsorted(s["child_indptr"].long(), i, right=True) - 1
        j = i - s["child_indptr"].long()[f]
        src = s["kv_indices"].long()[s["kv_indptr"].long()[s["parents_t"].long()[f]] + j]
        past = j - s["keep_t"].long()[f]
        new = past >= 0
        table = src.clone()
        table[new] = s["fresh"].long()[s["fresh_indptr"].long()[f[new]] + past[new]]
        s["pool_t"][table[new]] = s["pool_t"][src[new]]
        table = table.to(torch.int32)
    return s["pool_t"].view(torch.float8_e4m3fn), table


def _run_compact(s):
    if own:
        from split_kv_mla_gb300 import mla
        table, live = mla.mla_cache_compact(s["pool_t"], s["kv_indices"], workspace_t=s["ws"])
    else:
        idx = s["kv_indices"].long()
        n = s["pool"]
        used = torch.zeros(n + 1, dtype=torch.bool, device="cuda")
        used[torch.where(idx >= 0, idx, torch.full_like(idx, n))] = True
        used = used[:n]
        count = used.sum()
        at = torch.arange(n, device="cuda")
        holes, tail = at[~used & (at < count)], at[used & (at >= count)]
        to = at.clone()
        to[tail] = holes
        s["pool_t"][holes] = s["pool_t"][tail]
        table = torch.where(idx >= 0, to[idx.clamp(min=0)], idx).to(torch.int32)
        live = count.to(torch.int32).view(1)
    return s["pool_t"].view(torch.float8_e4m3fn), table, live


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "prefix":
        rows = case["batch"] * case["q_len"] * case["heads"]
        mean = (case["lo"] + case["hi"]) / 2
        keys = case["prefix"] + case["batch"] * mean
        return dict(bytes=keys * (576 + 4) + rows * (2 * 576 + 2 * 512 + 4),
                    flops=2.0 * rows * (case["prefix"] + mean) * (576 + 512))
    if op == "append":
        T, H, W, D = case["tokens"], case["heads"], case["width"], case["q_cols"]
        on = T - case["holes"]
        return dict(bytes=on * 3 * W + T * (256 + 8) + T * H * D * 4,
                    flops=6.0 * (on * W + T * H * (D if case["q_norm"] else 64)))
    if op == "fork":
        table = case["children"] * case["length"]
        rows = case["children"] * (case["length"] - case["keep"])
        return dict(bytes=rows * 2 * case["width"] + table * 8 + rows * 4, flops=0)
    n, live = case["pool"], case["live"]
    moved = live * (n - live) / n   # live rows expected at or past the live count
    table = live + max(1, live // 8) * min(case["requests"] - 1, 7) + 5
    return dict(bytes=moved * 2 * case["width"] + table * 8, flops=0)


# ---- the definitions in 64 bits -------------------------------------------------------------

def _e4m3(byte):
    """The value of an e4m3fn code: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    sign = -1.0 if byte & 0x80 else 1.0
    e, m = (byte >> 3) & 15, byte & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))


def _values(codes):
    table = torch.tensor([_e4m3(b) for b in range(256)], dtype=torch.float64, device=codes.device)
    return table[codes.int()]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prefix":
        B, Q, H = case["batch"], case["q_len"], case["heads"]
        outs, lses = [], []
        for b in range(B):
            n = int(s["seq_lens"][b])
            i0 = int(s["kv_indptr"][b])
            slots = torch.cat([s["prefix_indices"], s["kv_indices"][i0:i0 + n]]).long()
            k = _values(s["pool_t"][slots]) * KV_SCALE
            for t in range(Q):
                seen = max(0, len(slots) - Q + t + 1)
                q = torch.cat([s["q_lat"][b * Q + t], s["q_pe"][b * Q + t]], -1).double()
                if seen == 0:
                    outs.append(torch.zeros(H, 512, dtype=torch.float64, device=q.device))
                    lses.append(torch.full((H,), -math.inf, dtype=torch.float64, device=q.device))
                    continue
                logits = q @ k[:seen].T * 576.0 ** -0.5
                outs.append(torch.softmax(logits, -1) @ k[:seen, :512])
                lses.append(torch.logsumexp(logits, -1) / math.log(2.0))
        return torch.stack(outs), torch.stack(lses)
    if op == "append":
        W, D, T = case["width"], case["q_cols"], case["tokens"]
        n = 512
        kv = s["kv"].double()
        rms = (kv[:, :n].pow(2).sum(-1, keepdim=True) / n + EPS).sqrt()
        kv[:, :n] = kv[:, :n] / rms * s["kv_weight"].double()
        q = s["q"].double()
        if case["q_norm"]:
            q = q / (q.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * s["q_weight"].double()
        cs = s["cos_sin"].double()[s["positions"].long()]
        turn = torch.complex(cs[:, :32], cs[:, 32:])
        def rot(x, turn):
            if case["half"]:
                z = torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous()) * turn
                return torch.cat([z.real, z.imag], -1)
            z = torch.view_as_complex(x.contiguous().view(*x.shape[:-1], 32, 2)) * turn
            return torch.view_as_real(z).reshape(x.shape)
        kv[:, W - 64:] = rot(kv[:, W - 64:], turn)
        pool = _values(s["pool_t"])
        keep = (s["slots"] >= 0).nonzero()[:, 0]
        pool[s["slots"].long()[keep]] = (kv[keep] / KV_SCALE).clamp(-448, 448)
        q_pe = rot(q[..., D - 64:], turn[:, None])
        return (pool, q_pe) if D == 64 else (pool, q_pe, q[..., :D - 64])
    if op == "fork":
        pool, tables = _values(s["pool_t"]), []
        for f in range(case["children"]):
            p, k = int(s["parents_t"][f]), int(s["keep_t"][f])
            mine = s["kv_indices"][int(s["kv_indptr"][p]):int(s["kv_indptr"][p + 1])].long()
            fresh = s["fresh"][int(s["fresh_indptr"][f]):int(s["fresh_indptr"][f + 1])].long()
            pool[fresh] = _values(s["pool_t"][mine[k:]])
            tables.append(torch.cat([mine[:k], fresh]))
        return pool, torch.cat(tables).to(torch.int32)
    named = torch.unique(s["kv_indices"][s["kv_indices"] >= 0].long())
    count = named.numel()
    low = torch.zeros(count, dtype=torch.bool, device="cuda")
    low[named[named < count]] = True
    holes, tail = (~low).nonzero()[:, 0], named[named >= count]
    pool = _values(s["pool_t"])
    pool[holes] = _values(s["pool_t"][tail])
    table = s["kv_indices"].clone()
    moved = table >= count
    table[moved] = holes[torch.searchsorted(tail, table[moved].long())].to(torch.int32)
    return pool, table, torch.tensor([count], dtype=torch.int32, device="cuda")
