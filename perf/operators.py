"""The paged-cache operators, case by case, in plain torch operations and as the library's calls.

One page pool serves many requests: K and V are [pages][kv_heads][page_size][head_dim], `bounds` holds each
full page's smallest and largest key value per channel, and a block table gives each request's pages in order.

  tables   which pages and slots a step's new tokens take, from the requests' lengths
  write    a step's key and value rows into their slots, and the bounds of the pages that fill
  sparse   attention of each query over its newest pages and the best of the others by their bounds
  prefix   attention of a batch over a prefix that all its requests share and over their own pages
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of a serving batch: every request gets one token, a sixteenth of them a new page
        dict(name="tables decode 64", op="tables", requests=64, before=2304, new=1, page=16),
        # prompts of a large batch admitted in one go
        dict(name="tables prompts 4096", op="tables", requests=4096, before=1024, new=256, page=16),
        # one decode step of the grouped-query layer with 64 requests
        dict(name="write decode 64", op="write", requests=64, rows=64, before=2304, kv_heads=8, d=128, page=32, dtype="bf16"),
        # ragged prompts of 16 requests, some of which continue a partly filled page
        dict(name="write prompts 32768", op="write", requests=16, rows=32768, before=100, kv_heads=8, d=128, page=64, dtype="bf16"),
        # the smallest attention call: the small fp32 layer after its prompt, 4 query heads to 4 caches
        dict(name="sparse f32 d64", op="sparse", requests=1, tokens=1, context=192, kv_heads=4, groups=1, d=64, page=16, budget=8, recent=2, dtype="f32"),
        # one request with a 32768-token context and a cache per query head, budget 4096 tokens
        dict(name="sparse 1x32k", op="sparse", requests=1, tokens=1, context=32768, kv_heads=32, groups=1, d=128, page=16, budget=256, recent=128, dtype="bf16"),
        # several tokens a request (drafted tokens that are checked together), head_dim 64, odd sizes
        dict(name="sparse drafts d64", op="sparse", requests=7, tokens=5, context=9001, kv_heads=2, groups=8, d=64, page=64, budget=17, recent=3, dtype="bf16"),
        # a serving batch of long grouped-query contexts, budget 4096 tokens
        dict(name="sparse 64x24k", op="sparse", requests=64, tokens=1, context=24576, kv_heads=8, groups=4, d=128, page=32, budget=128, recent=8, dtype="bf16"),
        # a small fp32 batch behind a common instruction
        dict(name="prefix f32 d64", op="prefix", requests=16, tokens=1, prefix=2048, context=128, kv_heads=4, groups=1, d=64, page=16, dtype="f32"),
        # the grouped-query layer: 8 requests behind a 2048-token prompt
        dict(name="prefix 8x2k", op="prefix", requests=8, tokens=1, prefix=2048, context=410, kv_heads=8, groups=4, d=128, page=16, dtype="bf16"),
        # a cache per query head, 200 requests behind 8000 shared tokens
        dict(name="prefix 200x8k", op="prefix", requests=200, tokens=1, prefix=8000, context=256, kv_heads=32, groups=1, d=128, page=32, dtype="bf16"),
        # 64 requests that ask about the same 32768-token document
        dict(name="prefix 64x32k", op="prefix", requests=64, tokens=1, prefix=32768, context=512, kv_heads=8, groups=8, d=128, page=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "write", "sparse", "prefix"])
    page, d = rng.choice([16, 32, 64, 128]), rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    if op == "tables":
        n = _log(rng, 1, 4096)
        return dict(op=op, requests=n, before=_log(rng, 1, 4096), new=_log(rng, 1, min(2048, max(1, 4096 * 256 // n))), page=page)
    if op == "write":
        heads = rng.choice([1, 2, 4, 8, 32])
        rows = _log(rng, 1, 32768 * 8 * 128 * 2 // (heads * d * size) if heads * d * size > 2048 else 32768)
        return dict(op=op, requests=max(1, rows // _log(rng, 1, 512)), rows=rows, before=_log(rng, 1, 1000), kv_heads=heads, d=d, page=page, dtype=dtype)
    if op == "sparse":
        heads, groups = rng.choice([(1, 16), (2, 8), (3, 5), (4, 1), (8, 4), (8, 8), (32, 1)])
        context = _log(rng, 64, 32768)
        pages = max(2, context // page)
        budget = min(_log(rng, 2, max(3, pages)), max(2, 4096 // page))
        tokens = rng.choice([1, 1, 2, 3, 7])
        most = 64 * 8 * 4096 * 256 // (heads * tokens * min(context, budget * page) * d * size)
        return dict(op=op, requests=_log(rng, 1, max(1, min(64, most))), tokens=tokens, context=context, kv_heads=heads, groups=groups, d=d, page=page,
                    budget=budget, recent=rng.randint(1, max(1, budget // 2)), dtype=dtype)
    heads, groups = rng.choice([(1, 16), (2, 8), (3, 5), (4, 1), (8, 4), (8, 8), (32, 1)])
    prefix, tokens = _log(rng, 16, 32768), rng.choice([1, 1, 2, 5])
    flops = 64 * 64 * 32768 if dtype == "bf16" else 64 * 64 * 2048  # queries times keys: the largest listed case, and what fp32 arithmetic does in about its time
    most = max(1, flops // (heads * groups * tokens * prefix))
    return dict(op=op, requests=_log(rng, 1, min(256 // tokens, most)), tokens=tokens, prefix=prefix, context=_log(rng, 8, 512), kv_heads=heads, groups=groups, d=d,
                page=page, dtype=dtype)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(requests, lo, hi, gen):
    return torch.randint(lo, hi + 1, (requests,), device="cuda", generator=gen, dtype=torch.int32)


def _table(owned, width, perm):
    """[requests][width] block table: request i owns `owned[i]` pages, in the order of `perm`; -1 where it owns none."""
    start = torch.cumsum(owned, 0) - owned
    w = torch.arange(width, device="cuda")
    at = start[:, None] + w[None]
    return torch.where(w[None] < owned[:, None], perm[at.clamp(max=perm.numel() - 1)], -1).to(torch.int32)


def _pool(pages, heads, page, d, dtype, gen):
    """Keys that lie around a centre of their page's own, and values."""
    k = torch.randn(pages, heads, page, d, device="cuda", dtype=dtype, generator=gen)
    k += torch.randn(pages, heads, 1, d, device="cuda", dtype=dtype, generator=gen)
    return k, torch.randn(pages, heads, page, d, device="cuda", dtype=dtype, generator=gen)


def prepare(case, seed):
    gen, op, ps = _gen(seed), case["op"], case["page"]
    n, s = case["requests"], dict(case)
    if op == "tables":
        before = _lengths(n, 0, case["before"], gen)
        new = _lengths(n, 1, max(1, 2 * case["new"] - 1), gen)
        width = -(-(case["before"] + 2 * case["new"]) // ps)
        owned = (before + ps - 1) // ps
        pages = n * width + 1
        perm = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
        table = _table(owned, width, perm)
        cap = n * max(1, 2 * case["new"] - 1)
        empty = lambda k: torch.empty(k, device="cuda", dtype=torch.int32)  # noqa: E731
        s.update(before=before, new=new, table=table, after=empty(n), start=empty(n + 1), seq=empty(cap), pos=empty(cap), slot=empty(cap), status=empty(4))
        used = torch.zeros(pages, device="cuda", dtype=torch.bool)
        used[table[table >= 0].long()] = True
        s["free"] = perm[~used[perm.long()]].contiguous()  # the pages that no request owns
        return s
    dtype, heads, d = DTYPES[case["dtype"]], case["kv_heads"], case["d"]
    if op == "write":
        rows = case["rows"]
        cuts = torch.randint(0, rows + 1, (n - 1,), device="cuda", generator=gen) if n != rows else torch.arange(1, rows, device="cuda")
        ends = torch.cat([cuts.sort().values, torch.tensor([rows], device="cuda")])
        new = torch.diff(ends, prepend=torch.zeros(1, device="cuda", dtype=ends.dtype))
        before = _lengths(n, 0, case["before"], gen).long()
        owned = (before + new + ps - 1) // ps
        pages = n * (-(-case["before"] // ps) + 1) + -(-rows // ps)
        perm = torch.randperm(pages, device="cuda", generator=gen)
        r = torch.arange(rows, device="cuda")
        seq = torch.searchsorted(ends, r, right=True)
        pos = before[seq] + r - (ends - new)[seq]
        slot = perm[(torch.cumsum(owned, 0) - owned)[seq] + pos // ps] * ps + pos % ps
        K, V = _pool(pages, heads, ps, d, dtype, gen)
        k, v = (torch.randn(rows, heads, d, device="cuda", dtype=dtype, generator=gen) for _ in range(2))
        s.update(k=k, v=v, slot=slot.to(torch.int32), K=K, V=V, bounds=torch.zeros(pages, heads, 2, d, device="cuda", dtype=dtype))
        return s
    t, g = case["tokens"], case["groups"]
    context = case["context"]
    length = _lengths(n, max(t, context // 2), max(t, context), gen)
    width = -(-max(t, context) // ps)
    owned = (length + ps - 1) // ps
    shared = -(-case["prefix"] // ps) if op == "prefix" else 0
    perm = torch.randperm(n * width + shared, device="cuda", generator=gen)
    K, V = _pool(perm.numel(), heads, ps, d, dtype, gen)
    r = torch.arange(n * t, device="cuda", dtype=torch.int32)
    q = torch.randn(n * t, heads * g, d, device="cuda", dtype=dtype, generator=gen)
    s.update(q=q, K=K, V=V, table=_table(owned, width, perm[shared:]), row_seq=r // t, row_pos=length[(r // t).long()] - t + r % t, out=torch.empty_like(q),
             scale=d ** -0.5)
    if op == "sparse":
        s["bounds"] = torch.stack([K.amin(2), K.amax(2)], 2)
        s["picked"] = torch.empty(n * t, heads, case["budget"], device="cuda", dtype=torch.int32)
    else:
        s["shared"] = perm[:shared].to(torch.int32)
    return s


def _run_own(s):
    from kv_cache_eviction_h2o_gb300 import binding as L
    stream = torch.cuda.current_stream()
    if s["op"] == "tables":
        L.h2o_page_tables(s["before"], s["new"], s["free"], s["page"], s["table"], s["after"], s["start"], s["seq"], s["pos"], s["slot"], s["status"], stream)
        return [s[x] for x in ("table", "after", "start", "seq", "pos", "slot", "status")]
    if s["op"] == "write":
        L.h2o_page_write(s["k"], s["v"], s["slot"], s["K"], s["V"], s["bounds"], stream)
        return [s["K"], s["V"], s["bounds"]]
    if s["op"] == "sparse":
        L.h2o_page_attend(s["q"], s["row_seq"], s["row_pos"], s["K"], s["V"], s["bounds"], s["table"], s["budget"], s["recent"], s["scale"], s["out"], s["picked"], stream)
        return [s["out"], s["picked"]]
    work = torch.empty(L.h2o_prefix_work_bytes(s["q"].shape[0], s["kv_heads"], s["groups"], s["d"], s["prefix"], L.H2O_BF16 if s["dtype"] == "bf16" else L.H2O_F32),
                       device="cuda", dtype=torch.uint8)
    L.h2o_prefix_attend(s["q"], s["row_seq"], s["row_pos"], s["K"], s["V"], s["shared"], s["prefix"], s["table"], s["scale"], s["out"], work, stream)
    return [s["out"]]


def run(s):
    if own:
        return _run_own(s)
    return {"tables": _tables, "write": _write, "sparse": _sparse, "prefix": _prefix}[s["op"]](s)


def _tables(s):
    before, new, free, ps, table = s["before"], s["new"], s["free"], s["page"], s["table"]
    n, width, cap = before.numel(), table.shape[1], s["slot"].numel()
    after = before + new
    owned, want = (before + ps - 1) // ps, (after + ps - 1) // ps
    need = want - owned
    first = torch.cumsum(need, 0) - need
    w = torch.arange(width, device="cuda", dtype=torch.int32)[None]
    at = (first - owned)[:, None] + w
    fresh = (w >= owned[:, None]) & (w < want[:, None])
    table = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table)
    ends = torch.cumsum(new, 0).to(torch.int32)
    start = torch.cat([ends.new_zeros(1), ends])
    r = torch.arange(cap, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(ends, r, right=True, out_int32=True)
    live, i = seq < n, seq.clamp(max=n - 1).long()
    pos = before[i] + r - start[i]
    slot = table[i, (pos // ps).clamp(0, width - 1).long()] * ps + pos % ps
    seq, pos, slot = (torch.where(live, x, -1) for x in (seq, pos, slot))
    status = torch.stack([ends[-1], need.sum().to(torch.int32), after.max(), torch.zeros_like(ends[0])])
    return [table, after, start, seq, pos, slot, status]


def _write(s):
    ps, K, V, bounds = s["page"], s["K"], s["V"], s["bounds"]
    slot = s["slot"].long()
    page, at = slot // ps, slot % ps
    K[page, :, at] = s["k"]
    V[page, :, at] = s["v"]
    filled = torch.zeros(K.shape[0], device="cuda", dtype=torch.int32).index_add_(0, page, (at == ps - 1).to(torch.int32)) > 0
    bounds.copy_(torch.where(filled[:, None, None, None], torch.stack([K.amin(2), K.amax(2)], 2), bounds))
    return [K, V, bounds]


def _attend(q, logits, values):
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - top)
    return (p / p.sum(-1, keepdim=True)) @ values


def _sparse(s):
    q, K, V, ps, budget, recent = s["q"], s["K"], s["V"], s["page"], s["budget"], s["recent"]
    rows, heads, d = q.shape[0], K.shape[1], K.shape[3]
    table, pos = s["table"][s["row_seq"].long()].long(), s["row_pos"].long()
    width = table.shape[1]
    table = table.clamp(min=0)
    qh = q.view(rows, heads, -1, d)
    # scores in 64 bits: a page next to the border is in or out by its last bits
    q64 = qh.double()
    w = torch.stack([q64.clamp(max=0).sum(2), q64.clamp(min=0).sum(2)], 2).view(rows, heads, 2 * d, 1)
    b = s["bounds"][table].permute(0, 2, 1, 3, 4).reshape(rows, heads, width, 2 * d)
    score = (b.double() @ w)[..., 0]
    page = torch.arange(width, device="cuda")
    pages = (pos // ps + 1)[:, None, None]
    score = torch.where(page < pages - recent, score, torch.where(page < pages, math.inf, -math.inf))
    score, at = torch.sort(score, dim=-1, descending=True, stable=True)  # ties go to the lowest page
    take = min(budget, width)
    at = torch.where(score[..., :take] > -math.inf, at[..., :take], width).sort(-1).values
    live = at < width
    real = table[torch.arange(rows, device="cuda")[:, None, None], at.clamp(max=width - 1)]
    h = torch.arange(heads, device="cuda")[None, :, None]
    keys, vals = (x[real, h].reshape(rows, heads, take * ps, d).float() for x in (K, V))
    key_pos = (at[..., None] * ps + torch.arange(ps, device="cuda")).view(rows, heads, 1, take * ps)
    logits = torch.where(key_pos <= pos[:, None, None, None], (qh.float() @ keys.transpose(-1, -2)) * s["scale"], -math.inf)
    out = _attend(qh, logits, vals).view(q.shape).to(q.dtype)
    picked = torch.full((rows, heads, budget), -1, device="cuda", dtype=torch.int32)
    picked[..., :take] = torch.where(live, at, -1).to(torch.int32)
    return [out, picked]


def _prefix(s):
    q, K, V, ps, prefix = s["q"], s["K"], s["V"], s["page"], s["prefix"]
    rows, heads, d = q.shape[0], K.shape[1], K.shape[3]
    table = s["table"][s["row_seq"].long()].long().clamp(min=0)
    qh = q.view(rows, heads, -1, d).float()
    shared = [x[s["shared"].long()].transpose(0, 1).reshape(heads, -1, d)[:, :prefix].float() for x in (K, V)]
    mine = [x[table].transpose(1, 2).reshape(rows, heads, -1, d).float() for x in (K, V)]
    key_pos = torch.arange(mine[0].shape[2], device="cuda")
    seen = key_pos <= s["row_pos"][:, None, None, None]
    a = qh.transpose(0, 1).reshape(heads, -1, d) @ shared[0].transpose(-1, -2)
    a = a.view(heads, rows, -1, prefix).transpose(0, 1) * s["scale"]
    b = torch.where(seen, (qh @ mine[0].transpose(-1, -2)) * s["scale"], -math.inf)
    top = torch.maximum(a.amax(-1, keepdim=True), b.amax(-1, keepdim=True))
    a, b = torch.exp(a - top), torch.exp(b - top)
    total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    a = (a.transpose(0, 1).reshape(heads, -1, prefix) @ shared[1]).view(heads, rows, -1, d).transpose(0, 1)
    return [((a + b @ mine[1]) / total).reshape(q.shape).to(q.dtype)]


def work(case):
    n, ps = case["requests"], case["page"]
    if case["op"] == "tables":
        rows, cap, taken = n * case["new"], n * max(1, 2 * case["new"] - 1), n * case["new"] / ps
        # lengths, free pages and the last page of each request in; new pages, lengths, starts and three maps out
        return {"bytes": 8 * n + 4 * taken + 4 * n + 4 * taken + 4 * n + 4 * (n + 1) + 12 * cap + 16, "flops": rows}
    size, heads, d = (2 if case["dtype"] == "bf16" else 4), case["kv_heads"], case["d"]
    if case["op"] == "write":
        rows = case["rows"]
        return {"bytes": 4 * rows * heads * d * size + 4 * rows + rows / ps * heads * 2 * d * size, "flops": 2 * rows * heads * d}
    t, g, context = case["tokens"], case["groups"], case["context"]
    rows, mean = n * t, 0.75 * max(t, context)
    io = 2 * rows * heads * g * d * size + 8 * rows
    if case["op"] == "sparse":
        pages = mean / ps
        others = max(0.0, pages - case["recent"]) if pages > case["budget"] else 0.0
        keys = min(case["budget"] * ps, mean)
        # a request's own tokens may read the same pages: each is read once at best
        return {"bytes": io + n * heads * (others * 2 * d * size + min(t * keys, mean) * 2 * d * size) + 4 * rows * heads * case["budget"],
                "flops": rows * heads * (4 * g * d * keys + 4 * d * others)}
    keys = case["prefix"] + mean
    return {"bytes": io + heads * case["prefix"] * 2 * d * size + n * heads * mean * 2 * d * size, "flops": 4 * rows * heads * g * d * keys}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None  # whole numbers
    if case["op"] == "write":
        return _exact_write(s)
    rows, ps, heads, g, d = s["q"].shape[0], s["page"], s["kv_heads"], s["groups"], s["d"]
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    seq, pos, table = s["row_seq"].tolist(), s["row_pos"].tolist(), s["table"].cpu().numpy()
    for r in range(rows):
        mine = table[seq[r]][: pos[r] // ps + 1]
        q = s["q"][r].double().view(heads, g, d)
        if case["op"] == "sparse":
            lists = [_best(s, q[h], mine, h) for h in range(heads)]
        else:
            lists = [np.arange(len(mine))] * heads
        for h in range(heads):
            real = torch.from_numpy(mine[lists[h]]).long().cuda()
            at = torch.from_numpy((lists[h][:, None] * ps + np.arange(ps)).reshape(-1)).cuda()
            keys, vals = (x[real, h].reshape(-1, d)[at <= pos[r]].double() for x in (s["K"], s["V"]))
            if case["op"] == "prefix":
                first = s["shared"].long()
                keys, vals = (torch.cat([x[first, h].reshape(-1, d)[: s["prefix"]].double(), y]) for x, y in ((s["K"], keys), (s["V"], vals)))
            z = torch.einsum("gd,kd->gk", q[h], keys) * s["scale"]
            e = torch.exp(z - z.max(1, keepdim=True).values)
            out[r, h * g : (h + 1) * g] = torch.einsum("gk,kd->gd", e, vals) / e.sum(1)[:, None]
    return [out, None] if case["op"] == "sparse" else [out]


def _best(s, q, mine, h):
    """The pages one query row of one cache head reads: the newest, and the best of the others."""
    n, budget, recent = len(mine), s["budget"], s["recent"]
    if n <= budget:
        return np.arange(n)
    b = s["bounds"][torch.from_numpy(mine[: n - recent]).long().cuda(), h].double()
    most = torch.maximum(q[:, None, :] * b[None, :, 0], q[:, None, :] * b[None, :, 1])
    score = most.sum((0, 2)).cpu().numpy()
    best = np.lexsort((np.arange(n - recent), -score))[: budget - recent]
    return np.concatenate([np.sort(best), np.arange(n - recent, n)])


def _exact_write(s):
    K, V, bounds, ps = s["K"].double(), s["V"].double(), s["bounds"].double(), s["page"]
    slot = s["slot"].long()
    flat = [x.transpose(1, 2).reshape(-1, *x.shape[1::2]) for x in (K, V)]
    for x, y in zip(flat, (s["k"], s["v"])):
        x.index_copy_(0, slot, y.double())
    K, V = (x.view(-1, ps, *x.shape[1:]).transpose(1, 2) for x in flat)
    last = slot[slot % ps == ps - 1] // ps
    bounds[last, :, 0], bounds[last, :, 1] = K[last].min(2).values, K[last].max(2).values
    return [K, V, bounds]
