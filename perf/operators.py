"""Cases of the paged K/V cache operators: the page plan, the cache append and the attention over the cache.

``listed()`` names the cases, ``prepare`` makes what a serving loop has in hand before a call, ``run`` is one call (the
framework's where ``own`` is true, else the operator's plain form in elementary torch operations), ``exact`` the
definition in 64 bits."""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# the largest listed attention cases: multiply-adds (times 2) and bytes a drawn case stays below
MOST_FLOPS = 1.0e12
MOST_BYTES = 2.0e9


def lengths(case):
    """(cached, new) tokens of every request: fixed by the case, spread over its ranges (logarithmically)."""
    r = random.Random(case["lens"])

    def one(lo, hi):
        return lo if hi <= lo else min(hi, max(lo, round(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1))
    ctx, new = [], []
    for i in range(case["nreq"]):
        long = i < case["long"]  # the requests that bring a chunk; the others bring one token
        ctx.append(one(case["ctx_lo"], case["ctx_hi"]))
        new.append(one(case["new_lo"], case["new_hi"]) if long else 1)
    if case["nreq"] > 1:  # in any order, as a scheduler leaves them
        order = list(range(case["nreq"]))
        r.shuffle(order)
        ctx, new = [ctx[i] for i in order], [new[i] for i in order]
    return ctx, new


def listed():
    gqa = {"hq": 32, "hkv": 8, "hd": 128, "dtype": "bf16"}
    return [
        # the plan of one decode step of a batch: the smallest call, once per generated token
        {"name": "plan decode", "op": "plan", "nreq": 64, "long": 0, "ctx_lo": 100, "ctx_hi": 32768, "new_lo": 1,
         "new_hi": 1, "page": 64, "lens": 1},
        # the plan of a large prefill: many prompts and continued chunks, small pages
        {"name": "plan prefill", "op": "plan", "nreq": 256, "long": 250, "ctx_lo": 0, "ctx_hi": 16384, "new_lo": 100,
         "new_hi": 4096, "page": 16, "lens": 2},
        # K/V of one decode step into the cache
        {"name": "append decode", "op": "append", "nreq": 64, "long": 0, "ctx_lo": 100, "ctx_hi": 2048, "new_lo": 1,
         "new_hi": 1, "page": 64, "lens": 3, **gqa},
        # K/V of long prompts into the cache
        {"name": "append prompts", "op": "append", "nreq": 9, "long": 9, "ctx_lo": 0, "ctx_hi": 300, "new_lo": 4096,
         "new_hi": 16384, "page": 64, "lens": 4, **gqa},
        # the framework's other type, one K/V head, small pages, an odd count
        {"name": "append f32", "op": "append", "nreq": 5, "long": 4, "ctx_lo": 3, "ctx_hi": 900, "new_lo": 700,
         "new_hi": 2500, "page": 16, "lens": 5, "hq": 8, "hkv": 1, "hd": 64, "dtype": "f32"},
        # one token each for a few short requests: the latency of a call
        {"name": "decode short", "op": "attn", "nreq": 4, "long": 0, "ctx_lo": 300, "ctx_hi": 1024, "new_lo": 1,
         "new_hi": 1, "page": 16, "lens": 6, **gqa},
        # a decode step of a batch of uneven requests: the ordinary serving step
        {"name": "decode batch", "op": "attn", "nreq": 64, "long": 0, "ctx_lo": 2000, "ctx_hi": 16384, "new_lo": 1,
         "new_hi": 1, "page": 64, "lens": 7, **gqa},
        # one token of the longest sequence the bench runs, and a second one: few rows, a very long axis
        {"name": "decode long", "op": "attn", "nreq": 2, "long": 0, "ctx_lo": 200000, "ctx_hi": 262143, "new_lo": 1,
         "new_hi": 1, "page": 128, "lens": 8, **gqa},
        # a chunk of a long prompt over what is cached of it
        {"name": "chunk long", "op": "attn", "nreq": 1, "long": 1, "ctx_lo": 64000, "ctx_hi": 64000, "new_lo": 900,
         "new_hi": 900, "page": 64, "lens": 9, **gqa},
        # whole prompts of different lengths, nothing cached before
        {"name": "prompts", "op": "attn", "nreq": 6, "long": 6, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 1500,
         "new_hi": 4100, "page": 16, "lens": 10, **gqa},
        # decodes and short chunks in one batch, head dim 64, five query heads to a K/V head
        {"name": "mixed", "op": "attn", "nreq": 33, "long": 7, "ctx_lo": 0, "ctx_hi": 8192, "new_lo": 2,
         "new_hi": 300, "page": 32, "lens": 11, "hq": 20, "hkv": 4, "hd": 64, "dtype": "bf16"},
        # the framework's other type: a chunk in fp32, as many K/V heads as query heads
        {"name": "chunk f32", "op": "attn", "nreq": 2, "long": 2, "ctx_lo": 2000, "ctx_hi": 4096, "new_lo": 200,
         "new_hi": 512, "page": 16, "lens": 12, "hq": 8, "hkv": 8, "hd": 64, "dtype": "f32"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    while True:
        op = rng.choice(["plan", "append", "attn", "attn", "attn"])
        c = {"op": op, "page": rng.choice([16, 32, 64, 128, 256]), "lens": rng.randrange(1 << 30)}
        if op == "plan":
            c["nreq"] = log(1, 512)
            c["long"] = rng.randint(0, c["nreq"])
            c["ctx_lo"], c["ctx_hi"] = 0, log(100, 32768)
            c["new_lo"], c["new_hi"] = 1, log(2, 8192)
        else:
            kind = rng.choice(["decode", "chunk", "prompt", "mixed"])
            c["hkv"] = rng.choice([1, 2, 4, 8])
            c["hq"] = c["hkv"] * rng.choice([1, 2, 3, 4, 5, 7, 8])
            c["hd"], c["dtype"] = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "bf16", "f32"])
            c["nreq"] = log(1, 128) if kind in ("decode", "mixed") else log(1, 8)
            c["long"] = {"decode": 0, "mixed": c["nreq"] // 3}.get(kind, c["nreq"])
            c["ctx_lo"], c["ctx_hi"] = (0, 0) if kind == "prompt" else (0, log(100, 131072))
            c["new_lo"], c["new_hi"] = 1, log(2, 4096)
        ctx, new = lengths(c)
        if sum(new) > 262144:
            continue
        w = work(c)
        pad = c["nreq"] * max(new) * max(x + y for x, y in zip(ctx, new)) * c.get("hq", 1)
        dense = c["nreq"] * max(x + y for x, y in zip(ctx, new)) * c.get("hkv", 1) * c.get("hd", 1) * 8
        if op == "attn" and (w["flops"] > MOST_FLOPS * (0.02 if c["dtype"] == "f32" else 1) or pad > 2.5e9):
            continue
        if w["bytes"] > MOST_BYTES or dense > 2e10:
            continue
        return c


class State:
    pass


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    s = State()
    ctx, new = lengths(case)
    ps, nreq = case["page"], case["nreq"]
    s.case, s.page, s.nreq, s.T = case, ps, nreq, sum(new)
    old = [-(-c // ps) for c in ctx]
    total = [-(-(c + n) // ps) for c, n in zip(ctx, new)]
    s.width = max(total) + 3            # the table is a little wider than the longest request
    s.pages = sum(total) + 5            # and the cache a little larger than what is in use
    ids = torch.randperm(s.pages, generator=h, dtype=torch.int32)
    held = old if case["op"] == "plan" else total
    table = torch.full((nreq, s.width), -1, dtype=torch.int32)
    col = torch.arange(s.width)[None, :] < torch.tensor(held)[:, None]
    table[col] = ids[:sum(held)]
    s.table = table.cuda()
    s.new_host, s.max_new = new, max(new)
    s.ctx = torch.tensor(ctx, dtype=torch.int32).cuda()
    s.new = torch.tensor(new, dtype=torch.int32).cuda()
    s.cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    s.kv = s.ctx + s.new
    if case["op"] == "plan":
        # the free list: two pages of earlier steps are taken, the rest is free
        s.free = torch.cat([ids[:2], ids[sum(held):]]).cuda()
        s.head = torch.tensor([2], dtype=torch.int32).cuda()
        return s
    hq, hkv, hd, dt = case["hq"], case["hkv"], case["hd"], DTYPES[case["dtype"]]
    s.G, s.scale = hq // hkv, 1.0 / math.sqrt(hd)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)
    s.k_cache, s.v_cache = normal(s.pages, hkv, ps, hd), normal(s.pages, hkv, ps, hd)
    if case["op"] == "append":
        s.k, s.v = normal(s.T, hkv, hd), normal(s.T, hkv, hd)
        pos = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)])
        req = torch.repeat_interleave(torch.arange(nreq), torch.tensor(new))
        s.slots = (table[req, pos // ps] * ps + pos % ps).to(torch.int32).cuda()
        return s
    s.q = normal(s.T, hq, hd) * 1.5     # scores of a standard deviation of 1.5
    s.max_kv = max(c + n for c, n in zip(ctx, new))
    # a serving loop keeps one workspace for all of its calls
    s.workspace = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    return s


def plain_plan(s):
    ps = s.page
    ctx, new = s.ctx.long(), s.new.long()
    total = ctx + new
    old, every = (ctx + ps - 1) // ps, (total + ps - 1) // ps
    fresh = every - old
    first = torch.cumsum(fresh, 0) - fresh + s.head.long()
    col = torch.arange(s.width, device="cuda")[None, :]
    at = first[:, None] + col - old[:, None]
    is_new = (col >= old[:, None]) & (col < every[:, None])
    page = s.free[at.clamp(0, s.free.numel() - 1)]
    s.table.copy_(torch.where(is_new, torch.where(at < s.free.numel(), page, -1), s.table))
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(new, 0)])
    t = torch.arange(s.T, device="cuda")
    req = torch.searchsorted(cu, t, right=True) - 1
    pos = ctx[req] + t - cu[req]
    entry = s.table[req, pos // ps]
    slots = torch.where(entry >= 0, entry * ps + (pos % ps).int(), -1)
    counts = torch.stack([cu[-1], s.head[0].long() + fresh.sum(), (slots < 0).sum(), total.max()]).int()
    return [s.table, slots, cu.int(), total.int(), counts]


def plain_append(s):
    slots = s.slots.long()
    page, at = slots // s.page, slots % s.page
    s.k_cache[page, :, at] = s.k
    s.v_cache[page, :, at] = s.v
    return [s.k_cache, s.v_cache]


def plain_attn(s):
    nreq, hkv, G, hd = s.nreq, s.case["hkv"], s.G, s.case["hd"]
    used = -(-s.max_kv // s.page)
    pages = s.table[:, :used].clamp(min=0).long()
    k = s.k_cache[pages].float().transpose(1, 2).reshape(nreq, hkv, used * s.page, hd)
    v = s.v_cache[pages].float().transpose(1, 2).reshape(nreq, hkv, used * s.page, hd)
    j = torch.arange(s.max_new, device="cuda")
    rows = (s.cu[:-1, None] + j).clamp(max=s.T - 1).long()                 # (request, token)
    q = s.q[rows].float().reshape(nreq, s.max_new, hkv, G, hd).permute(0, 2, 1, 3, 4)
    scores = q.reshape(nreq, hkv, s.max_new * G, hd) @ k.transpose(2, 3)
    scores = scores.mul_(s.scale).view(nreq, hkv, s.max_new, G, used * s.page)
    limit = torch.minimum((s.kv - s.new)[:, None] + j + 1, s.kv[:, None])  # keys a token sees
    hidden = torch.arange(used * s.page, device="cuda") >= limit[:, :, None]
    scores.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    m = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(nreq, hkv, s.max_new * G, -1) @ v).view(nreq, hkv, s.max_new, G, hd)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, m + total.log(), -math.inf)
    t = torch.arange(s.T, device="cuda")
    req = torch.searchsorted(s.cu, t, right=True) - 1
    tok = t - s.cu[req]
    out = o[req, :, tok].reshape(s.T, hkv * G, hd).to(s.q.dtype)
    return [out, lse[req, :, tok].reshape(s.T, hkv * G)]


def run(s):
    op = s.case["op"]
    if own:
        import sequence_long_context_zigzag_gb300 as usp
    if op == "plan":
        if own:
            slots, cu, kv, counts = usp.usp_page_plan(s.ctx, s.new, s.free, s.head, s.table, s.page, s.pages, s.T)
            return [s.table, slots, cu, kv, counts]
        return plain_plan(s)
    if op == "append":
        if own:
            usp.usp_cache_append(s.k, s.v, s.k_cache, s.v_cache, s.slots)
            return [s.k_cache, s.v_cache]
        return plain_append(s)
    if own:
        out, lse = usp.usp_paged_attn(s.q, s.k_cache, s.v_cache, s.table, s.cu, s.kv, s.max_new,
                                      workspace=s.workspace)
        return [out, lse]
    return plain_attn(s)


def work(case):
    ctx, new = lengths(case)
    ps, nreq, T = case["page"], case["nreq"], sum(new)
    if case["op"] == "plan":
        fresh = sum(-(-(c + n) // ps) - -(-c // ps) for c, n in zip(ctx, new))
        # lengths, free pages and head read; table entries, slots, cu, kv and counts written; the page a
        # request's first new token shares with its cached ones read
        shared = sum(1 for c, n in zip(ctx, new) if n and c % ps)
        return {"bytes": 4 * (2 * nreq + fresh + 1 + fresh + T + nreq + 1 + nreq + 4 + shared), "flops": 0}
    es = 4 if case["dtype"] == "f32" else 2
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    if case["op"] == "append":
        return {"bytes": 4 * T * hkv * hd * es + 4 * T, "flops": 0}
    keys = sum(c + n for c, n in zip(ctx, new))
    pages = sum(-(-(c + n) // ps) for c, n in zip(ctx, new))
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    return {"bytes": es * (2 * T * hq * hd + 2 * keys * hkv * hd) + 4 * (T * hq + pages + 2 * nreq + 1),
            "flops": 4 * hq * hd * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None                     # whole numbers only
    ctx, new = lengths(case)
    ps = case["page"]
    if case["op"] == "append":
        k, v = s.k_cache.double(), s.v_cache.double()
        flat_k, flat_v = k.transpose(1, 2).reshape(-1, *s.k.shape[1:]), v.transpose(1, 2).reshape(-1, *s.v.shape[1:])
        flat_k.index_copy_(0, s.slots.long(), s.k.double())
        flat_v.index_copy_(0, s.slots.long(), s.v.double())
        shape = (s.pages, ps, *s.k.shape[1:])
        return [flat_k.view(shape).transpose(1, 2).contiguous(), flat_v.view(shape).transpose(1, 2).contiguous()]
    out = torch.zeros(s.T, case["hq"], case["hd"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(s.T, case["hq"], dtype=torch.float64, device="cuda")
    t0 = 0
    for i, (c, n) in enumerate(zip(ctx, new)):
        pos = torch.arange(c + n, device="cuda")
        page, at = s.table[i, pos // ps].long(), pos % ps
        for head in range(case["hkv"]):
            k, v = s.k_cache[page, head, at].double(), s.v_cache[page, head, at].double()
            for a in range(0, n, 512):
                b = min(n, a + 512)
                heads = slice(head * s.G, (head + 1) * s.G)
                q = s.q[t0 + a:t0 + b, heads].double()
                e = torch.einsum("tgd,sd->tgs", q, k) / math.sqrt(case["hd"])
                seen = pos[None, :] <= c + torch.arange(a, b, device="cuda")[:, None]
                e = e.masked_fill(~seen[:, None, :], -math.inf)
                z = torch.logsumexp(e, -1)
                out[t0 + a:t0 + b, heads] = torch.einsum("tgs,sd->tgd", torch.exp(e - z[..., None]), v)
                lse[t0 + a:t0 + b, heads] = z
        t0 += n
    return [out, lse]
