"""Cases of the position rotation and of the 4-bit paged cache: the rotation of whole sequences with its gradient, the
append with the rotation on the way, the append into a 4-bit cache and the attention over one.

``listed()`` names the cases, ``prepare`` makes what a user's program has in hand before a call, ``run`` is one call (the
framework's where ``own`` is true, else the operator's plain form in elementary torch operations), ``exact`` the
definition in 64 bits."""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# the largest listed cases: multiply-adds (times 2) and bytes a drawn case stays below
MOST_FLOPS = 9.0e11
MOST_BYTES = 1.7e9


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


def samples(case):
    """Cumulative lengths of the samples packed into a sequence."""
    r = random.Random(case["lens"])
    cuts = sorted(r.sample(range(1, case["L"]), case["nseq"] - 1))
    return [0] + cuts + [case["L"]]


def listed():
    gqa = {"hq": 32, "hkv": 8, "hd": 128, "dtype": "bf16"}
    return [
        # a layer's q and k of a long training sequence, rotated, and their gradients rotated back
        {"name": "rope train", "op": "rope", "bs": 1, "L": 32768, "nseq": 1, "rot": 128, "pairs": False, "lens": 1, **gqa},
        # the other type and pairing, packed samples of odd lengths, only half of each head rotated: a small step
        {"name": "rope packed", "op": "rope", "bs": 2, "L": 5001, "nseq": 7, "rot": 32, "pairs": True, "lens": 2, "hq": 6,
         "hkv": 2, "hd": 64, "dtype": "f32"},
        # q, K and V of one decode step: the smallest call, once per layer and generated token
        {"name": "append decode", "op": "append", "q4": False, "nreq": 64, "long": 0, "ctx_lo": 100, "ctx_hi": 2048,
         "new_lo": 1, "new_hi": 1, "page": 64, "lens": 3, "rot": 128, "pairs": False, **gqa},
        # q, K and V of long prompts
        {"name": "append prompts", "op": "append", "q4": False, "nreq": 7, "long": 7, "ctx_lo": 0, "ctx_hi": 300,
         "new_lo": 4096, "new_hi": 16384, "page": 64, "lens": 4, "rot": 128, "pairs": False, **gqa},
        # a decode step whose cache is held in 4 bits
        {"name": "append q4 decode", "op": "append", "q4": True, "nreq": 64, "long": 0, "ctx_lo": 100, "ctx_hi": 2048,
         "new_lo": 1, "new_hi": 1, "page": 64, "lens": 5, "rot": 128, "pairs": False, **gqa},
        # K (rotated before) and V of long prompts into a 4-bit cache
        {"name": "append q4 prompts", "op": "append", "q4": True, "nreq": 9, "long": 9, "ctx_lo": 0, "ctx_hi": 300,
         "new_lo": 4096, "new_hi": 16384, "page": 16, "lens": 6, "rot": 0, "pairs": False, **gqa},
        # one token each for a few short requests: the latency of a call
        {"name": "q4 decode short", "op": "attn", "nreq": 4, "long": 0, "ctx_lo": 300, "ctx_hi": 1024, "new_lo": 1,
         "new_hi": 1, "page": 16, "lens": 7, **gqa},
        # a decode step of a batch of uneven requests: the ordinary serving step
        {"name": "q4 decode batch", "op": "attn", "nreq": 64, "long": 0, "ctx_lo": 2000, "ctx_hi": 32768, "new_lo": 1,
         "new_hi": 1, "page": 64, "lens": 8, **gqa},
        # one token of the longest sequence the bench runs, and a second one: few rows, a very long axis
        {"name": "q4 decode long", "op": "attn", "nreq": 2, "long": 0, "ctx_lo": 200000, "ctx_hi": 262143, "new_lo": 1,
         "new_hi": 1, "page": 128, "lens": 9, **gqa},
        # a chunk of a long prompt over what is cached of it
        {"name": "q4 chunk long", "op": "attn", "nreq": 1, "long": 1, "ctx_lo": 48000, "ctx_hi": 48000, "new_lo": 1000,
         "new_hi": 1000, "page": 64, "lens": 10, **gqa},
        # decodes and short chunks in one batch, head dim 64, five query heads to a K/V head
        {"name": "q4 mixed", "op": "attn", "nreq": 33, "long": 7, "ctx_lo": 0, "ctx_hi": 8192, "new_lo": 2,
         "new_hi": 300, "page": 32, "lens": 11, "hq": 20, "hkv": 4, "hd": 64, "dtype": "bf16"},
        # fp32 queries: a few tokens each to be checked at once, as many K/V heads as query heads
        {"name": "q4 f32", "op": "attn", "nreq": 6, "long": 6, "ctx_lo": 2000, "ctx_hi": 9000, "new_lo": 3,
         "new_hi": 12, "page": 16, "lens": 12, "hq": 8, "hkv": 8, "hd": 64, "dtype": "f32"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    while True:
        op = rng.choice(["rope", "append", "append", "attn", "attn", "attn"])
        c = {"op": op, "lens": rng.randrange(1 << 30), "hd": rng.choice([64, 128])}
        c["hkv"] = rng.choice([1, 2, 4, 8])
        c["hq"] = c["hkv"] * rng.choice([1, 2, 3, 4, 5, 7, 8])
        c["dtype"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
        if op != "attn":
            c["rot"], c["pairs"] = rng.choice([c["hd"], c["hd"], c["hd"] // 2, 48]), rng.choice([False, False, True])
        if op == "rope":
            c["bs"], c["L"] = rng.choice([1, 1, 2, 3]), log(50, 60000)
            c["nseq"] = rng.choice([1, rng.randint(2, 20)])
        else:
            c["page"] = rng.choice([16, 32, 64, 128, 256])
            kind = rng.choice(["decode", "chunk", "prompt", "mixed"])
            c["nreq"] = log(1, 128) if kind in ("decode", "mixed") else log(1, 8)
            c["long"] = {"decode": 0, "mixed": c["nreq"] // 3}.get(kind, c["nreq"])
            most = log(100, 131072 if op == "attn" else 4096)
            c["ctx_lo"], c["ctx_hi"] = (0, 0) if kind == "prompt" else (rng.choice([0, most // 4]), most)
            c["new_hi"] = log(2, 8192)
            c["new_lo"] = rng.choice([1, c["new_hi"] // 2])
            if op == "append":
                c["q4"] = rng.choice([False, True])
                if c["q4"] and rng.random() < 0.3:
                    c["rot"] = 0
            ctx, new = lengths(c)
            if sum(new) > 131072:
                continue
            pad = c["nreq"] * max(new) * max(x + y for x, y in zip(ctx, new)) * c["hq"]
            dense = c["nreq"] * max(x + y for x, y in zip(ctx, new)) * c["hkv"] * c["hd"] * 8
            if op == "attn" and (pad > 2.5e9 or dense > 1.2e10):
                continue
        w = work(c)
        if w["bytes"] > MOST_BYTES or w["flops"] > MOST_FLOPS * (0.02 if c["dtype"] == "f32" else 1):
            continue
        return c


class State:
    pass


def rope_table(n, rot):
    """cos and sin of every position's angles, side by side, fp32: what a model keeps."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    s = State()
    hq, hkv, hd, dt = case["hq"], case["hkv"], case["hd"], DTYPES[case["dtype"]]
    s.case = case

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)
    if case["op"] == "rope":
        bs, L = case["bs"], case["L"]
        s.table = rope_table(L, case["rot"])
        s.q, s.k = normal(bs, L, hq, hd).requires_grad_(), normal(bs, L, hkv, hd).requires_grad_()
        s.dq, s.dk = normal(bs, L, hq, hd), normal(bs, L, hkv, hd)
        s.cu = torch.tensor(samples(case), dtype=torch.int32).cuda() if case["nseq"] > 1 else None
        return s
    ctx, new = lengths(case)
    ps, nreq = case["page"], case["nreq"]
    s.page, s.nreq, s.T = ps, nreq, sum(new)
    total = [-(-(c + n) // ps) for c, n in zip(ctx, new)]
    s.width = max(total) + 3            # the table is a little wider than the longest request
    s.pages = sum(total) + 5            # and the cache a little larger than what is in use
    ids = torch.randperm(s.pages, generator=h, dtype=torch.int32)
    blocks = torch.full((nreq, s.width), -1, dtype=torch.int32)
    blocks[torch.arange(s.width)[None, :] < torch.tensor(total)[:, None]] = ids[:sum(total)]
    s.blocks = blocks.cuda()
    s.max_new, s.max_kv = max(new), max(c + n for c, n in zip(ctx, new))
    s.new = torch.tensor(new, dtype=torch.int32).cuda()
    s.cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    s.kv = torch.tensor(ctx, dtype=torch.int32).cuda() + s.new

    def codes():  # two codes a byte, as rounded normal values give them
        lo, hi = ((torch.randn(s.pages, hkv, ps, hd // 2, generator=g, device="cuda", dtype=torch.bfloat16) * 2.6)
                  .round().clamp(-8, 7).to(torch.int8) for _ in range(2))
        return ((lo & 15) | (hi << 4)).view(torch.uint8)

    def scales():  # 0.19 to 0.7
        return torch.randint(140, 156, (s.pages, hkv, ps, hd // 32), generator=g, device="cuda", dtype=torch.uint8)
    if case["op"] == "append":
        s.q, s.k, s.v = normal(s.T, hq, hd), normal(s.T, hkv, hd), normal(s.T, hkv, hd)
        pos = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)])
        req = torch.repeat_interleave(torch.arange(nreq), torch.tensor(new))
        s.slots = (blocks[req, pos // ps] * ps + pos % ps).to(torch.int32).cuda()
        s.table = rope_table(s.max_kv, case["rot"]) if case["rot"] else None
        if case["q4"]:
            s.k_cache, s.v_cache, s.k_scales, s.v_scales = codes(), codes(), scales(), scales()
        else:
            s.k_cache, s.v_cache = normal(s.pages, hkv, ps, hd), normal(s.pages, hkv, ps, hd)
        return s
    s.G, s.scale = hq // hkv, 1.0 / math.sqrt(hd)
    s.k_cache, s.v_cache, s.k_scales, s.v_scales = codes(), codes(), scales(), scales()
    s.q = normal(s.T, hq, hd) * 1.5     # scores of a standard deviation of about 1.5
    # a serving loop keeps one workspace for all of its calls
    s.workspace = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------
def rotated(x, c, s, rot, pairs):
    """x (..., H, hd) in 32 bits, rotated by the angles whose cos and sin (..., rot / 2) these are."""
    c, s = c.unsqueeze(-2), s.unsqueeze(-2)
    y = x.float().clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    u, v = x[..., a].float(), x[..., b].float()
    y[..., a] = u * c - v * s
    y[..., b] = v * c + u * s
    return y


def plain_rope(s):
    case, t = s.case, s.table
    pos = torch.arange(case["L"], device="cuda")
    if s.cu is not None:
        pos = pos - s.cu[torch.searchsorted(s.cu, pos, right=True) - 1]
    half = case["rot"] // 2
    c, n = t[pos, :half], t[pos, half:]
    fore = [rotated(x.detach(), c, n, case["rot"], case["pairs"]).to(x.dtype) for x in (s.q, s.k)]
    back = [rotated(x, c, -n, case["rot"], case["pairs"]).to(x.dtype) for x in (s.dq, s.dk)]
    return fore + back


def quantised(x):
    """Codes (two a byte) and scale bytes of x (..., hd), 32 bits: groups of 32, scales (8 + b % 8) 2^(b // 8 - 23), the
    smallest with 7.5 scale >= the group's largest value; codes x / scale to the nearest whole number, ties to even."""
    x = x.unflatten(-1, (-1, 32))
    byte = torch.arange(256, device="cuda")
    scale = ((byte << 20) + (107 << 23)).to(torch.int32).view(torch.float32)
    b = torch.searchsorted(scale * 7.5, x.abs().amax(-1)).clamp(max=255)
    u = (x.double() / scale[b].double()[..., None]).round().clamp(-8, 7).to(torch.int8) & 15
    # of each 8 values, the even ones in the low nibbles of the 32-bit word's low half, the odd ones of its high half
    u = u.flatten(-2).unflatten(-1, (-1, 4, 2)).transpose(-1, -2).reshape(*x.shape[:-2], -1, 2)
    return (u[..., 0] | (u[..., 1] << 4)).view(torch.uint8), b.to(torch.uint8)


def plain_append(s):
    case = s.case
    q, k, v = None, s.k.float(), s.v.float()
    if case["rot"]:
        t = torch.arange(s.T, device="cuda")
        req = torch.searchsorted(s.cu, t, right=True) - 1
        pos = (s.kv[req] - s.cu[req + 1] + t).long()
        half = case["rot"] // 2
        c, n = s.table[pos, :half], s.table[pos, half:]
        q = rotated(s.q, c, n, case["rot"], case["pairs"]).to(s.q.dtype)
        k = rotated(s.k, c, n, case["rot"], case["pairs"])
    slots = s.slots.long()
    page, at = slots // s.page, slots % s.page
    if case["q4"]:
        s.k_cache[page, :, at], s.k_scales[page, :, at] = quantised(k)
        s.v_cache[page, :, at], s.v_scales[page, :, at] = quantised(v)
    else:
        s.k_cache[page, :, at] = k.to(s.k.dtype)
        s.v_cache[page, :, at] = s.v
    return appended(s, q)


def appended(s, q):
    """The state after an append. The bytes of a 4-bit cache are whole numbers that the operator's definition fixes
    (ties and scales too), so they are compared as such: what they stand for is then the same."""
    state = [s.k_cache, s.v_cache] + ([s.k_scales, s.v_scales] if s.case["q4"] else [])
    return state if q is None else [q] + state


def values(codes, scales):
    """What a 4-bit cache's codes and scale bytes stand for, in 32 bits."""
    hd = codes.shape[-1] * 2
    u = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], hd // 8, 2, 4).transpose(-1, -2)
    c = ((u.view(torch.int8) ^ 8) - 8).reshape(*codes.shape[:-1], hd // 32, 32)
    scale = ((scales.int() << 20) + (107 << 23)).view(torch.float32)
    return (c * scale[..., None]).flatten(-2)


def plain_attn(s):
    nreq, hkv, G, hd = s.nreq, s.case["hkv"], s.G, s.case["hd"]
    used = -(-s.max_kv // s.page)
    pages = s.blocks[:, :used].clamp(min=0).long()
    k = values(s.k_cache[pages], s.k_scales[pages]).transpose(1, 2).reshape(nreq, hkv, used * s.page, hd)
    v = values(s.v_cache[pages], s.v_scales[pages]).transpose(1, 2).reshape(nreq, hkv, used * s.page, hd)
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
    op, case = s.case["op"], s.case
    if own:
        import sequence_long_context_zigzag_gb300 as usp
    if op == "rope":
        if own:
            q, k = usp.UspRopeFunction.apply(s.q, s.k, s.table, None, s.cu, case["pairs"])
            dq, dk = torch.autograd.grad((q, k), (s.q, s.k), (s.dq, s.dk))
            return [q, k, dq, dk]
        return plain_rope(s)
    if op == "append":
        if not own:
            return plain_append(s)
        q = None
        if not case["rot"]:
            usp.usp_cache_append_q4(s.k, s.v, s.k_cache, s.v_cache, s.k_scales, s.v_scales, s.slots)
        elif case["q4"]:
            q = usp.usp_rope_append(s.q, s.k, s.v, s.k_cache, s.v_cache, s.slots, s.table, s.cu, s.kv,
                                    k_scales=s.k_scales, v_scales=s.v_scales, interleaved=case["pairs"])
        else:
            q = usp.usp_rope_append(s.q, s.k, s.v, s.k_cache, s.v_cache, s.slots, s.table, s.cu, s.kv,
                                    interleaved=case["pairs"])
        return appended(s, q)
    if own:
        out, lse = usp.usp_paged_attn_q4(s.q, s.k_cache, s.v_cache, s.k_scales, s.v_scales, s.blocks, s.cu, s.kv,
                                         s.max_new, workspace=s.workspace)
        return [out, lse]
    return plain_attn(s)


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    if case["op"] == "rope":
        T = case["bs"] * case["L"]
        row = (hq + hkv) * hd
        return {"bytes": 4 * T * row * es + 4 * case["L"] * case["rot"], "flops": 6 * T * (hq + hkv) * case["rot"]}
    ctx, new = lengths(case)
    ps, nreq, T = case["page"], case["nreq"], sum(new)
    cached = hd // 2 + hd // 32  # bytes of a 4-bit row
    if case["op"] == "append":
        rotation = 4 * case["rot"] + 2 * hq * hd * es if case["rot"] else 0
        return {"bytes": T * (2 * hkv * (hd * es + (cached if case["q4"] else hd * es)) + rotation + 4) +
                (4 * (2 * nreq + 1) if case["rot"] else 0), "flops": 3 * T * (hq + hkv) * case["rot"]}
    keys = sum(c + n for c, n in zip(ctx, new))
    pages = sum(-(-(c + n) // ps) for c, n in zip(ctx, new))
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    return {"bytes": es * 2 * T * hq * hd + 2 * keys * hkv * cached + 4 * (T * hq + pages + 2 * nreq + 1),
            "flops": 4 * hq * hd * pairs}


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------
def turned(x, table, pos, rot, pairs, back=False):
    """x (T, H, hd) as complex pairs times e^(i angle) (e^(-i angle) where `back`), from the fp32 table's cos and sin."""
    half = rot // 2
    z = torch.complex(table[pos, :half].double(), table[pos, half:].double() * (-1 if back else 1))[:, None, :]
    y = x.double().clone()
    if pairs:
        w = torch.view_as_complex(y[..., :rot].unflatten(-1, (half, 2)).contiguous()) * z
        y[..., :rot] = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(y[..., :half].contiguous(), y[..., half:rot].contiguous()) * z
        y[..., :half], y[..., half:rot] = w.real, w.imag
    return y


def exact_values(codes, scales):
    """(keys, hd) in 64 bits from the codes (keys, hd / 2) and scale bytes (keys, hd / 32) of a head."""
    word = codes.contiguous().view(torch.int32).long() & 0xffffffff      # 8 codes each
    e = torch.arange(8, device="cuda")
    code = (word[..., None] >> (4 * (e // 2 + 4 * (e % 2)))) & 15
    code = torch.where(code >= 8, code - 16, code).double().flatten(-2)
    b = scales.double()
    scale = (8 + b % 8) * torch.pow(torch.full_like(b, 2.0), torch.floor(b / 8) - 23)
    return code * scale.repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        pos = torch.arange(case["L"], device="cuda")
        if s.cu is not None:
            starts = torch.tensor(samples(case), device="cuda")
            pos = torch.cat([torch.arange(n, device="cuda") for n in (starts[1:] - starts[:-1]).tolist()])
        pos = pos.repeat(case["bs"])
        return [turned(x.detach().flatten(0, 1), s.table, pos, case["rot"], case["pairs"], i > 1).view(x.shape)
                for i, x in enumerate((s.q, s.k, s.dq, s.dk))]
    ctx, new = lengths(case)
    ps = case["page"]
    if case["op"] == "append":
        out = []
        k = s.k.double()
        if case["rot"]:
            pos = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)]).cuda()
            out = [turned(s.q, s.table, pos, case["rot"], case["pairs"])]
            k = turned(s.k, s.table, pos, case["rot"], case["pairs"])
        if case["q4"]:
            return out + [None] * 4 if out else None    # whole numbers
        for cache, x in ((s.k_cache, k), (s.v_cache, s.v.double())):
            y = cache.double().transpose(1, 2).contiguous()
            y.view(-1, *x.shape[1:]).index_copy_(0, s.slots.long(), x)
            out.append(y.transpose(1, 2).contiguous())
        return out
    out = torch.zeros(s.T, case["hq"], case["hd"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(s.T, case["hq"], dtype=torch.float64, device="cuda")
    t0 = 0
    for i, (c, n) in enumerate(zip(ctx, new)):
        pos = torch.arange(c + n, device="cuda")
        page, at = s.blocks[i, pos // ps].long(), pos % ps
        for head in range(case["hkv"]):
            k = exact_values(s.k_cache[page, head, at], s.k_scales[page, head, at])
            v = exact_values(s.v_cache[page, head, at], s.v_scales[page, head, at])
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
