"""Inputs and 64-bit definitions for the paged K/V cache tests (plain torch, none of the library)."""
import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # finfo(dtype).eps / 2


class Cache:
    """Caches of spare and shuffled pages holding ``reqs`` = [(keys, new tokens)]; every row that no
    request owns is NaN. ``interleave``: K and V as the two halves of one buffer's pages."""

    def __init__(self, reqs, hq, hkv, hd, ps, dtype, seed=0, interleave=False, device="cuda", qpad=0, spare=3,
                 v_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.reqs, self.hq, self.hkv, self.hd, self.ps, self.dtype = reqs, hq, hkv, hd, ps, dtype
        n = [max(n, 0) for _, n in reqs]
        kv = [k for k, _ in reqs]
        T = sum(n)
        pages = [-(-max(k, 0) // ps) for k in kv]
        num = sum(pages) + spare
        ids = torch.randperm(num, generator=g)
        width = max(pages + [0]) + 1
        table = torch.full((len(reqs), width), -1, dtype=torch.int32)
        nan = float("nan")
        buf = torch.full((num, 2, hkv, ps, hd), nan, dtype=dtype)
        self.k, self.v = [], []
        at = 0
        for i, (k, p) in enumerate(zip(kv, pages)):
            mine = ids[at:at + p]
            at += p
            table[i, :p] = mine.to(torch.int32)
            kk = torch.randn(max(k, 0), hkv, hd, generator=g).to(dtype)
            vv = (torch.randn(max(k, 0), hkv, hd, generator=g) * v_scale).to(dtype)
            self.k.append(kk)
            self.v.append(vv)
            for c in range(p):
                rows = min(ps, k - c * ps)
                buf[mine[c], 0, :, :rows] = kk[c * ps:c * ps + rows].transpose(0, 1)
                buf[mine[c], 1, :, :rows] = vv[c * ps:c * ps + rows].transpose(0, 1)
        wide = torch.randn(T, hq * hd + qpad, generator=g).mul(1.5).to(dtype).to(device)
        self.q = wide[:, :hq * hd].unflatten(1, (hq, hd))
        buf = buf.to(device)
        self.k_cache, self.v_cache = buf[:, 0], buf[:, 1]
        if not interleave:
            self.k_cache, self.v_cache = self.k_cache.contiguous(), self.v_cache.contiguous()
        self.table = table.to(device)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=device)
        self.kv = torch.tensor(kv, dtype=torch.int32, device=device)
        self.T, self.max_new = T, max(n + [0])

    def args(self):
        return self.q, self.k_cache, self.v_cache, self.table, self.cu, self.kv


def attention64(c, causal=True, scale=None):
    """(out, lse, out bound, lse bound) in 64 bits. The bounds are the kernels' own roundings, from the
    inputs: with A = sum_j p_j |v_j| (p the softmax weights),
      scores: an fp32 sum of hd products, |ds| <= hd 2^-24 scale max_j sum |q k|, plus 2^-21 for the
        scaled exponent, the exponential and the running-maximum rescales (relative errors of weights);
      weights and sums: n keys in fp32, n 2^-24; bf16 weights add half a step, 2^-8, each;
      the output adds half a step of its own type.
    A relative error e of every weight moves o by at most e (A + |o|) <= 2 e A (numerator and
    normaliser); the bf16 rounding of weights enters the numerator only."""
    dev = c.q.device
    G, hd = c.hq // c.hkv, c.hd
    scale = 1.0 / math.sqrt(hd) if scale is None else scale
    out = torch.zeros(c.T, c.hq, hd, dtype=torch.float64, device=dev)
    lse = torch.full((c.T, c.hq), -math.inf, dtype=torch.float64, device=dev)
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    half = HALF_STEP[c.dtype]
    t0 = 0
    for i, (kv, n) in enumerate(c.reqs):
        n = max(n, 0)
        if kv > 0 and n > 0:
            k, v = c.k[i].to(dev).double(), c.v[i].to(dev).double()
            q = c.q[t0:t0 + n].double().view(n, c.hkv, G, hd)
            s = torch.einsum("nhgd,khd->nhgk", q, k) * scale
            ab = torch.einsum("nhgd,khd->nhgk", q.abs(), k.abs()).amax(-1) * scale
            pos = torch.arange(n, device=dev) + kv - n
            seen = torch.arange(kv, device=dev)[None] <= (pos[:, None] if causal else torch.full_like(pos, kv)[:, None])
            s = s.masked_fill(~seen[:, None, None, :], -math.inf)
            any_ = seen.any(-1)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(torch.isfinite(z), z, torch.zeros_like(z))[..., None])
            o = torch.einsum("nhgk,khd->nhgd", p, v)
            A = torch.einsum("nhgk,khd->nhgd", p, v.abs())
            e = hd * 2.0 ** -24 * ab + 2.0 ** -21 + kv * 2.0 ** -24
            b = 2 * e[..., None] * A + half * o.abs() + (2.0 ** -8 * A if c.dtype == torch.bfloat16 else 0)
            lb = e + 2.0 ** -23 * z.abs()
            o, z = o * any_[:, None, None, None], torch.where(any_[:, None, None], z, -math.inf)
            out[t0:t0 + n], lse[t0:t0 + n] = o.reshape(n, c.hq, hd), z.reshape(n, c.hq)
            bo[t0:t0 + n] = b.reshape(n, c.hq, hd)
            bl[t0:t0 + n] = torch.where(any_[:, None, None], lb, 0.0).reshape(n, c.hq)
        t0 += n
    return out, lse, bo * 1.01 + 1e-30, bl * 1.01


def check_attention(c, out, lse, causal=True, scale=None):
    o, z, bo, bl = attention64(c, causal, scale)
    err = (out.double() - o).abs()
    assert not torch.isnan(err).any(), "NaN in out"
    assert (err <= bo).all(), f"out off by up to {(err / bo).max().item():.3g} bounds"
    fin = torch.isfinite(z)
    assert torch.equal(torch.isfinite(lse), fin) and (lse[~fin] == -math.inf).all(), "lse of empty rows"
    el = (lse.double() - z).abs()[fin]
    assert (el <= bl[fin]).all(), f"lse off by up to {(el / bl[fin]).max().item():.3g} bounds"


def plan_ref(ctx, new, free, head, table, ps, num_pages, max_tokens):
    """usp_page_plan by the definition, in Python integers."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    slots, cu, kv, lost = [], [0], [], 0
    for i, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(c, 0), max(n, 0)
        old, every = -(-c // ps), -(-(c + n) // ps)
        for col in range(old, every):
            page = free[head] if head < len(free) else -1
            head += 1
            first = sum(max(x, 0) for x in new[:i]) + col * ps - c   # the new token that opens the page
            if col < width and first < max_tokens:
                table[i][col] = page
        for pos in range(c, c + n):
            col = pos // ps
            page = table[i][col] if col < width else -1
            slots.append(page * ps + pos % ps if 0 <= page < num_pages else -1)
            lost += col >= width or page == -1 and col >= old or len(slots) > max_tokens
        cu.append(min(cu[-1] + n, max_tokens))
        kv.append(c + n)
    total = len(slots)
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    return table, slots, cu, kv, [total, head, lost, max(kv + [0])]
