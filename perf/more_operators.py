"""Prompts and quantised paged caches, case by case, in plain torch operations and as the library's calls.

A prompt's way into a cache of 8- or 4-bit codes, and the decode that reads it: its queries and keys get their rotary
positions, its rows attend to one another, its keys and values are written as codes with one fp32 scale a row, come
back as rows for a prompt that goes on later, or are read as codes by the attention of single tokens.

  rope    rotary positions of query and key rows
  prompt  causal attention over the packed rows of several requests, each behind the tokens it already has
  store   key and value rows into a quantised page pool, and what it then holds for them
  read    rows of a quantised page pool
  attend  attention of single tokens over the whole quantised caches of their requests
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of the grouped-query layer with 64 requests at far positions, whole heads, half layout
        dict(name="rope decode 64", op="rope", rows=64, heads=32, kv_heads=8, d=128, rot=128, form="half", factor=1.0, far=32768, dtype="bf16"),
        # the grouped-query layer's prompts (8 x 2048 tokens), interleaved pairs in half of each head, scaled for a longer context
        dict(name="rope prompts 16384", op="rope", rows=16384, heads=32, kv_heads=8, d=128, rot=64, form="pairs", factor=8.0, far=131072, dtype="bf16"),
        # the smallest prompt: the small fp32 layer's 128 tokens of 4 heads
        dict(name="prompt f32 128", op="prompt", requests=1, new=128, before=0, kv_heads=4, groups=1, d=64, dtype="f32"),
        # the grouped-query layer's 8 prompts of up to 2048 tokens, of unequal lengths
        dict(name="prompt 8x2048", op="prompt", requests=8, new=2048, before=0, kv_heads=8, groups=4, d=128, dtype="bf16"),
        # a long prompt in parts: 2048 more tokens behind the 30000 that are already there, a cache per query head
        dict(name="prompt 2048 behind 30000", op="prompt", requests=1, new=2048, before=30000, kv_heads=32, groups=1, d=128, dtype="bf16"),
        # one decode step of the grouped-query layer with 64 requests, 8 bits
        dict(name="store decode 64", op="store", rows=64, kv_heads=8, d=128, page=32, bits=8, dtype="bf16"),
        # prompts of a serving batch, 4 bits
        dict(name="store prompts 32768", op="store", rows=32768, kv_heads=8, d=128, page=64, bits=4, dtype="bf16"),
        # a short fp32 context, read back for the next turn's prompt
        dict(name="read f32 777", op="read", rows=777, kv_heads=4, d=64, page=16, bits=8, dtype="f32"),
        # the context behind a long prompt's next part
        dict(name="read 32768", op="read", rows=32768, kv_heads=32, d=128, page=32, bits=4, dtype="bf16"),
        # the smallest attention call: the small fp32 layer after its prompt
        dict(name="attend f32 d64", op="attend", requests=1, tokens=1, context=192, kv_heads=4, groups=1, d=64, page=16, bits=8, dtype="f32"),
        # one request with a 32768-token context and a cache per query head, 8 bits
        dict(name="attend 1x32k", op="attend", requests=1, tokens=1, context=32768, kv_heads=32, groups=1, d=128, page=16, bits=8, dtype="bf16"),
        # a serving batch of long grouped-query contexts, 4 bits
        dict(name="attend 64x24k", op="attend", requests=64, tokens=1, context=24576, kv_heads=8, groups=4, d=128, page=32, bits=4, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(1, 16), (2, 8), (3, 5), (4, 1), (8, 4), (8, 8), (32, 1), (2, 7)]


def draw(rng):
    op = rng.choice(["rope", "prompt", "store", "read", "attend"])
    (heads, groups), d = rng.choice(HEADS), rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    if op == "rope":
        most = 16384 * 40 * 128 * 2 // ((groups + 1) * heads * d * size)
        return dict(op=op, rows=_log(rng, 1, min(65536, most)), heads=heads * groups, kv_heads=heads, d=d, rot=rng.choice([d, d, d // 2, d // 4, 24, 2]),
                    form=rng.choice(["half", "pairs"]), factor=rng.choice([1.0, 1.0, 4.0, 8.0, 32.0]), far=_log(rng, 16, 1 << 20), dtype=dtype)
    if op == "prompt":
        before = rng.choice([0, 0, _log(rng, 1, 32768)])
        cells = 32 * 2048 * 32000  # pairs of a query and a key, of all query heads, whatever the mask
        new = _log(rng, 1, 4096)
        new = max(1, min(new, cells // (heads * groups * (before + new))))
        most = max(1, min(64, cells // (heads * groups * new * (before + new))))
        return dict(op=op, requests=_log(rng, 1, most), new=new, before=before, kv_heads=heads, groups=groups, d=d, dtype=dtype)
    page, bits = rng.choice([16, 32, 64, 128]), rng.choice([8, 4])
    if op in ("store", "read"):
        return dict(op=op, rows=_log(rng, 1, min(65536, 32768 * 8 * 128 * 2 // (heads * d * size))), kv_heads=heads, d=d, page=page, bits=bits, dtype=dtype)
    context, tokens = _log(rng, 16, 32768), rng.choice([1, 1, 1, 2, 5])
    most = max(1, min(96, 64 * 24576 * 8 * 128 // (context * tokens * heads * d)))
    return dict(op=op, requests=_log(rng, 1, most), tokens=tokens, context=context, kv_heads=heads, groups=groups, d=d, page=page, bits=bits, dtype=dtype)


def _lengths(n, most):
    """n unequal lengths from `most` down to about half of it, odd ones among them; the same for every seed."""
    return [max(1, most - i * most // (2 * n) - i % 7) for i in range(n)] if most else [0] * n


def _frequencies(rot, factor):
    """Radians a position of each channel pair: base 10000, the slow ones divided by `factor`, by how often they turn in 4096 positions."""
    f = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    if factor == 1.0:
        return f
    kept = [min(1.0, max(0.0, (4096 * x / (2 * math.pi) - 1.0) / 31.0)) for x in f]
    return [x * ((1 - g) / factor + g) for x, g in zip(f, kept)]


def _starts(lengths):
    ends = [0]
    for n in lengths:
        ends.append(ends[-1] + n)
    return torch.tensor(ends, device="cuda", dtype=torch.int32)


def _shuffled(lengths, gen):
    return [lengths[i] for i in torch.randperm(len(lengths), generator=gen, device="cuda").tolist()]


def _codes(shape, bits, gen):
    """Random codes of a quantised pool, [..][d] int8, or two of 4 bits (offset by 8) in a byte, the even channel's low; and scales."""
    scale = torch.exp(0.4 * torch.randn(shape[:-1], device="cuda", generator=gen)) * (2.0 / (2 ** (bits - 1) - 1))
    if bits == 8:
        return torch.randint(-127, 128, shape, device="cuda", dtype=torch.int8, generator=gen), scale
    low, high = (torch.randint(1, 16, (*shape[:-1], shape[-1] // 2), device="cuda", dtype=torch.uint8, generator=gen) for _ in range(2))
    return low | high << 4, scale


def prepare(case, seed):
    gen, op, s = torch.Generator(device="cuda").manual_seed(seed), case["op"], dict(case)
    dtype, heads, d = DTYPES[case["dtype"]], case["kv_heads"], case["d"]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if op == "rope":
        # queries and keys are slices of one projection's output, and get their positions in new tensors
        rows, hq = case["rows"], case["heads"]
        both = randn(rows, hq + 2 * heads, d).to(dtype)
        q, k = both[:, :hq], both[:, hq : hq + heads]
        f = _frequencies(case["rot"], case["factor"])
        table = torch.tensor([round(x / (2 * math.pi) * 2.0**64) for x in f], dtype=torch.int64, device="cuda")  # 2^-64 turns a position
        s.update(q=q, k=k, frequency=torch.tensor(f, dtype=torch.float64, device="cuda"), table=table, amplitude=0.1 * math.log(case["factor"]) + 1.0,
                 row_pos=torch.randint(0, case["far"], (rows,), device="cuda", dtype=torch.int32, generator=gen), q_out=torch.empty(rows, hq, d, device="cuda", dtype=dtype),
                 k_out=torch.empty(rows, heads, d, device="cuda", dtype=dtype))
        return s
    if op == "prompt":
        n, g = case["requests"], case["groups"]
        new = _shuffled(_lengths(n, case["new"]), gen)
        before = _shuffled(_lengths(n, case["before"]), gen)
        rows, keys = sum(new), sum(new) + sum(before)
        s.update(q=randn(rows, heads * g, d).to(dtype), k=(randn(keys, heads, d) + randn(1, heads, d)).to(dtype), v=randn(keys, heads, d).to(dtype), q_start=_starts(new),
                 k_start=_starts([a + b for a, b in zip(new, before)]), scale=d**-0.5, out=torch.empty(rows, heads * g, d, device="cuda", dtype=dtype))
        return s
    ps, bits = case["page"], case["bits"]
    if op in ("store", "read"):
        rows = case["rows"]
        pages = -(-rows // ps) + 3
        perm = torch.randperm(pages, device="cuda", generator=gen)
        r = torch.arange(rows, device="cuda") + 5  # the first request continues a page
        s["slot"] = (perm[r // ps] * ps + r % ps).to(torch.int32)
        shape = (pages, heads, ps, d)
        if op == "store":
            loud = torch.exp(0.5 * randn(1, heads, d))  # channels differ in size
            s.update(k=(randn(rows, heads, d) * loud).to(dtype), v=randn(rows, heads, d).to(dtype))
            s["K"], s["V"] = (torch.zeros(pages, heads, ps, d * bits // 8, device="cuda", dtype=torch.int8 if bits == 8 else torch.uint8) for _ in range(2))
            s["kscale"], s["vscale"] = (torch.zeros(pages, heads, ps, device="cuda") for _ in range(2))
        else:
            (s["K"], s["kscale"]), (s["V"], s["vscale"]) = _codes(shape, bits, gen), _codes(shape, bits, gen)
        s["k_out"], s["v_out"] = (torch.empty(rows, heads, d, device="cuda", dtype=dtype) for _ in range(2))
        return s
    n, t, g, context = case["requests"], case["tokens"], case["groups"], case["context"]
    length = torch.tensor(_shuffled(_lengths(n, max(t, context)), gen), device="cuda", dtype=torch.int32).clamp(min=t)
    owned = (length + ps - 1) // ps
    width = -(-max(t, context) // ps)
    perm = torch.randperm(n * width, device="cuda", generator=gen)
    w = torch.arange(width, device="cuda")
    table = torch.where(w[None] < owned[:, None], perm[(torch.cumsum(owned, 0) - owned)[:, None] + torch.minimum(w[None], owned[:, None] - 1)], -1)
    shape = (n * width, heads, ps, d)
    (s["K"], s["kscale"]), (s["V"], s["vscale"]) = _codes(shape, bits, gen), _codes(shape, bits, gen)
    r = torch.arange(n * t, device="cuda", dtype=torch.int32)
    q = randn(n * t, heads * g, d).to(dtype)
    s.update(q=q, table=table.to(torch.int32), row_seq=r // t, row_pos=length[(r // t).long()] - t + r % t, scale=d**-0.5, out=torch.empty_like(q))
    return s


def _run_own(s):
    from kv_cache_eviction_h2o_gb300 import binding as L
    op = s["op"]
    if op == "rope":
        L.h2o_rope(s["q"], s["k"], s["row_pos"], s["table"], L.H2O_ROPE_HALF if s["form"] == "half" else L.H2O_ROPE_PAIRS, s["amplitude"], s["q_out"], s["k_out"])
        return [s["q_out"], s["k_out"]]
    if op == "prompt":
        L.h2o_prompt_attend(s["q"], s["k"], s["v"], s["q_start"], s["k_start"], s["scale"], s["out"])
        return [s["out"]]
    if op == "store":
        L.h2o_page_quant_write(s["k"], s["v"], s["slot"], s["K"], s["V"], s["kscale"], s["vscale"])
    if op in ("store", "read"):
        L.h2o_page_quant_read(s["K"], s["V"], s["kscale"], s["vscale"], s["slot"], s["k_out"], s["v_out"])
        return [s["k_out"], s["v_out"]] + ([s["kscale"], s["vscale"]] if op == "store" else [])
    L.h2o_page_quant_attend(s["q"], s["row_seq"], s["row_pos"], s["K"], s["V"], s["kscale"], s["vscale"], s["table"], s["scale"], s["out"])
    return [s["out"]]


def run(s):
    if own:
        return _run_own(s)
    return {"rope": _rope, "prompt": _prompt, "store": _store, "read": _read, "attend": _attend}[s["op"]](s)


def _rope(s):
    angle = s["row_pos"].double()[:, None, None] * s["frequency"]  # in 64 bits: far positions turn often
    cos, sin = (s["amplitude"] * torch.cos(angle)).float(), (s["amplitude"] * torch.sin(angle)).float()
    return [_rotated(s[x].float(), cos, sin, s["rot"], s["form"]).to(s[x].dtype) for x in ("q", "k")]


def _rotated(x, cos, sin, rot, form):
    turned, rest = x[..., :rot], x[..., rot:]
    if form == "half":
        a, b = turned[..., : rot // 2], turned[..., rot // 2 :]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = turned[..., 0::2], turned[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _softmax_sum(logits, values):
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    return (p @ values) / p.sum(-1, keepdim=True)


def _prompt(s):
    q, k, v, h, d = s["q"], s["k"], s["v"], s["kv_heads"], s["d"]
    nq, nk = torch.diff(s["q_start"]), torch.diff(s["k_start"])
    x = torch.arange(s["new"], device="cuda")
    y = torch.arange(s["new"] + s["before"], device="cuda")
    # requests padded to the longest: [requests, heads, rows, d]
    qi = (s["q_start"][:-1, None] + x).clamp(max=q.shape[0] - 1)
    ki = (s["k_start"][:-1, None] + y).clamp(max=k.shape[0] - 1)
    qs = q.float()[qi].view(*qi.shape, h, -1, d).permute(0, 2, 3, 1, 4)
    ks, vs = (z.float()[ki].permute(0, 2, 1, 3)[:, :, None] for z in (k, v))
    seen = y <= (nk - nq)[:, None, None] + x[:, None]
    logits = torch.where(seen[:, None, None], (qs @ ks.transpose(-1, -2)) * s["scale"], -math.inf)
    out = _softmax_sum(logits, vs).permute(0, 3, 1, 2, 4).reshape(*qi.shape, -1, d)
    return [out[x < nq[:, None]].to(q.dtype)]


def _quantised(x, bits):
    """Codes (in fp32) and scales of rows, in fp32 arithmetic: the rule is bit-exact."""
    amax = x.float().abs().amax(-1, keepdim=True)
    top = torch.full_like(amax, 2 ** (bits - 1) - 1)  # (a number over a tensor is the number times the rounded reciprocal)
    inv = torch.where(amax > 0, top / amax, torch.zeros_like(amax))
    return torch.round(x.float() * inv).clamp(-top, top), (amax / top)[..., 0]


def _unpacked(codes, bits):
    if bits == 8:
        return codes.float()
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8.0


def _store(s):
    ps, bits, slot = s["page"], s["bits"], s["slot"].long()
    page, at = slot // ps, slot % ps
    for x, pool, scales in (("k", "K", "kscale"), ("v", "V", "vscale")):
        code, scale = _quantised(s[x], bits)
        if bits == 4:
            code = code + 8
            code = code[..., 0::2] + 16 * code[..., 1::2]
        s[pool][page, :, at] = code.to(s[pool].dtype)
        s[scales][page, :, at] = scale
    return _read(s) + [s["kscale"], s["vscale"]]


def _read(s):
    ps, bits, slot = s["page"], s["bits"], s["slot"].long()
    page, at = slot // ps, slot % ps
    return [(_unpacked(s[pool][page, :, at], bits) * s[scales][page, :, at][..., None]).to(DTYPES[s["dtype"]]) for pool, scales in (("K", "kscale"), ("V", "vscale"))]


def _attend(s):
    q, ps, heads, d = s["q"], s["page"], s["kv_heads"], s["d"]
    rows = q.shape[0]
    table = s["table"].long().clamp(min=0)
    keys, vals = ((_unpacked(s[pool][table], s["bits"]) * s[scales][table][..., None]).transpose(1, 2).reshape(table.shape[0], heads, -1, d)
                  for pool, scales in (("K", "kscale"), ("V", "vscale")))
    # a request's tokens are adjacent rows: [requests, heads, tokens * groups, d]
    t = s["tokens"]
    qs = q.float().view(rows // t, t, heads, -1, d).transpose(1, 2)
    g = qs.shape[3]
    logits = (qs.reshape(rows // t, heads, t * g, d) @ keys.transpose(-1, -2)) * s["scale"]
    seen = torch.arange(keys.shape[2], device="cuda") <= s["row_pos"].view(-1, 1, t, 1, 1)
    logits = torch.where(seen.expand(-1, -1, -1, g, -1).reshape(rows // t, 1, t * g, -1), logits, -math.inf)
    return [_softmax_sum(logits, vals).view(rows // t, heads, t, g, d).transpose(1, 2).reshape(q.shape).to(q.dtype)]


def work(case):
    size, heads, d = (2 if case["dtype"] == "bf16" else 4), case["kv_heads"], case["d"]
    if case["op"] == "rope":
        rows, all_heads = case["rows"], case["heads"] + heads
        return {"bytes": 2 * rows * all_heads * d * size + 4 * rows + 4 * case["rot"], "flops": 3 * rows * all_heads * case["rot"]}
    if case["op"] == "prompt":
        new, before = _lengths(case["requests"], case["new"]), _lengths(case["requests"], case["before"])
        # (which length goes with which is the seed's: the mean of the earlier tokens stands for each)
        pairs = sum(n * (n + 1) / 2 + n * sum(before) / len(before) for n in new)
        hq = heads * case["groups"]
        return {"bytes": 2 * sum(new) * hq * d * size + 2 * (sum(new) + sum(before)) * heads * d * size, "flops": 4 * d * hq * pairs}
    code = d * case["bits"] // 8 + 4
    if case["op"] in ("store", "read"):
        rows = case["rows"]
        back = 2 * rows * heads * (d * size + code) + 4 * rows  # codes and scales in, rows out
        # (codes that were just written are in the nearest cache: they are counted once)
        return {"bytes": back + (2 * rows * heads * d * size if case["op"] == "store" else 0), "flops": rows * heads * d * (8 if case["op"] == "store" else 2)}
    rows, lengths = case["requests"] * case["tokens"], _lengths(case["requests"], max(case["tokens"], case["context"]))
    return {"bytes": 2 * rows * heads * case["groups"] * d * size + 8 * rows + sum(lengths) * heads * 2 * code,
            "flops": 4 * sum(lengths) * case["tokens"] * heads * case["groups"] * d}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "prompt": _exact_prompt, "store": _exact_store, "read": _exact_store, "attend": _exact_attend}[case["op"]](s)


def _exact_rope(s):
    turn = torch.polar(torch.full((), s["amplitude"], device="cuda", dtype=torch.float64), torch.outer(s["row_pos"].double(), s["frequency"]))[:, None]
    done, n = [], s["rot"] // 2
    for x in (s["q"], s["k"]):
        y = x.double()
        first, second = (slice(0, n), slice(n, 2 * n)) if s["form"] == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
        z = torch.complex(y[..., first], y[..., second]) * turn
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        done.append(y)
    return done


def _weighted(q, keys, vals, scale):
    z = torch.einsum("gd,kd->gk", q, keys) * scale
    e = torch.exp(z - z.max(1, keepdim=True).values)
    return torch.einsum("gk,kd->gd", e, vals) / e.sum(1)[:, None]


def _exact_prompt(s):
    qs, ks, g = s["q_start"].tolist(), s["k_start"].tolist(), s["groups"]
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    for i in range(s["requests"]):
        nq, nk = qs[i + 1] - qs[i], ks[i + 1] - ks[i]
        hidden = torch.ones(nq, nk, device="cuda", dtype=torch.bool).triu(nk - nq + 1)
        for h in range(s["kv_heads"]):
            keys, vals = (x[ks[i] : ks[i + 1], h].double() for x in (s["k"], s["v"]))
            for j in range(h * g, h * g + g):
                z = (s["q"][qs[i] : qs[i + 1], j].double() @ keys.T).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
                out[qs[i] : qs[i + 1], j] = torch.softmax(z, 1) @ vals
    return [out]


def _exact_store(s):
    """Codes by the rule's fp32 steps, each the rounding of a 64-bit result, and their values in 64 bits."""
    ps, top = s["page"], 2 ** (s["bits"] - 1) - 1
    at = torch.stack([s["slot"].long() // ps, s["slot"].long() % ps])
    rows, scales = [], []
    for x, pool, name in (("k", "K", "kscale"), ("v", "V", "vscale")):
        if s["op"] == "store":
            y = s[x].double()
            amax = torch.linalg.vector_norm(y, math.inf, dim=2)
            inv = torch.where(amax == 0, 0.0, (torch.full_like(amax, top) / amax).float().double())
            code = (y * inv[..., None]).float().double().round()
            scale = (amax / top).float().double()
            scales.append(s[name].double().index_put_((at[0][:, None], torch.arange(s["kv_heads"], device="cuda")[None], at[1][:, None]), scale))
        else:
            code, scale = s[pool].transpose(1, 2)[at[0], at[1]].long(), s[name].transpose(1, 2)[at[0], at[1]].double()
            if s["bits"] == 4:
                code = torch.stack([code % 16 - 8, code // 16 - 8], 3).reshape(*code.shape[:2], s["d"])
            code = code.double()
        rows.append(code * scale[..., None])
    return rows + scales


def _exact_attend(s):
    ps, heads, g, d = s["page"], s["kv_heads"], s["groups"], s["d"]
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    seq, pos = s["row_seq"].tolist(), s["row_pos"].tolist()
    for i in range(s["requests"]):
        mine = [r for r in range(len(seq)) if seq[r] == i]
        n = max(pos[r] for r in mine) + 1
        pages = s["table"][i, : -(-n // ps)].long()
        for h in range(heads):
            both = []
            for pool, name in (("K", "kscale"), ("V", "vscale")):
                code = s[pool][pages, h].reshape(len(pages) * ps, -1).long()
                if s["bits"] == 4:
                    code = torch.stack([code % 16 - 8, code // 16 - 8], 2).reshape(-1, d)
                both.append(code.double() * s[name][pages, h].reshape(-1, 1).double())
            for r in mine:
                out[r, h * g : h * g + g] = _weighted(s["q"][r, h * g : h * g + g].double(), *(x[: pos[r] + 1] for x in both), s["scale"])
    return [out]
