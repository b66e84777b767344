"""Inputs and definitions for the rotation and the 4-bit paged cache (plain torch and Python, none of the library)."""
import math
from fractions import Fraction

import numpy as np
import torch

NIBBLE = [e // 2 + 4 * (e % 2) for e in range(8)]      # the nibble of value e of a word's 8
SCALES = [Fraction(8 + (b & 7)) * Fraction(2) ** ((b >> 3) - 23) for b in range(256)]
SCALE64 = torch.tensor([float(s) for s in SCALES], dtype=torch.float64)


def values(codes, scales):
    """What codes (.., hd / 2) and scale bytes (.., hd / 32) stand for, in 64 bits."""
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (-1, 8)).long()
    c = nib[..., NIBBLE]
    c = torch.where(c >= 8, c - 16, c).flatten(-2).double()
    return c * SCALE64.to(codes.device)[scales.long()].repeat_interleave(32, -1)


def pack(c):
    """Codes (.., hd) of -8 .. 7 as bytes (.., hd / 2)."""
    u = (c.long() & 15).unflatten(-1, (-1, 8))
    nib = torch.empty_like(u)
    nib[..., NIBBLE] = u
    nib = nib.flatten(-2).unflatten(-1, (-1, 2))
    return (nib[..., 0] | nib[..., 1] << 4).to(torch.uint8)


def quantise(x):
    """(codes (.., hd / 2), scale bytes (.., hd / 32)) of fp32 or bf16 rows x (.., hd) by the definition. 64 bits hold
    a quotient of 24 by 4 bits far from any tie that it is not at."""
    x = x.double().unflatten(-1, (-1, 32))
    a = torch.where(x.isnan(), 0.0, x.abs()).amax(-1)
    b = torch.searchsorted(SCALE64.to(x.device) * 7.5, a).clamp(max=255)
    c = torch.where(x.isnan(), 0.0, x) / SCALE64.to(x.device)[b][..., None]
    return pack(c.clamp(-100, 100).round().clamp(-8, 7).flatten(-2)), b.to(torch.uint8)


def rope_table(n, rot, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate(x, table, pos, interleaved, inverse=False):
    """x (T, H, hd) rotated by the fp32 table's rows pos (-1: not at all): (fp32 with each operation rounded on its own,
    64 bits, bound of a result in x's type). Products and their sum are off by half a step each, then the result."""
    rot = table.shape[1]
    t = torch.cat([table, torch.cat([torch.ones(1, rot // 2), torch.zeros(1, rot // 2)], 1)])[pos.long()].to(x.device)
    c, s = t[:, None, :rot // 2], t[:, None, rot // 2:] * (-1 if inverse else 1)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    outs = []
    for y, c, s in ((x.float(), c, s), (x.double(), c.double(), s.double())):
        y = y.clone()
        u, v = y[..., a].clone(), y[..., b].clone()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
        outs.append(y)
    size = torch.zeros_like(outs[1])
    u, v, c, s = x[..., a].double().abs(), x[..., b].double().abs(), c.abs(), s.abs()
    size[..., a], size[..., b] = u * c + v * s, v * c + u * s
    half = torch.finfo(x.dtype).eps / 2
    return outs[0], outs[1], 2 * 2.0 ** -24 * size + half * outs[1].abs() + 1e-37


class Q4Cache:
    """4-bit caches of spare and shuffled pages holding ``reqs`` = [(keys, new tokens)]; rows that no request owns are
    random bytes with scales of any size. Fields as paged_ref.Cache's: k, v are what the requests' rows stand for."""

    def __init__(self, reqs, hq, hkv, hd, ps, dtype, seed=0, interleave=False, device="cuda", qpad=0, spare=3, wide=False):
        g = torch.Generator().manual_seed(seed)
        self.reqs, self.hq, self.hkv, self.hd, self.ps, self.dtype = reqs, hq, hkv, hd, ps, dtype
        n, kv = [max(n, 0) for _, n in reqs], [max(k, 0) for k, _ in reqs]
        pages = [-(-k // ps) for k in kv]
        num = sum(pages) + spare
        ids = torch.randperm(num, generator=g)
        table = torch.full((len(reqs), max(pages + [0]) + 1), -1, dtype=torch.int32)
        codes = torch.randint(0, 256, (num, 2, hkv, ps, hd // 2), generator=g, dtype=torch.uint8)
        scales = torch.randint(0, 256, (num, 2, hkv, ps, hd // 32), generator=g, dtype=torch.uint8)
        lo, hi = (100, 176) if wide else (140, 152)      # scales of 0.006 to 3, of 0.19 to 0.5
        self.k, self.v = [], []
        at = 0
        for i, (k, p) in enumerate(zip(kv, pages)):
            mine = ids[at:at + p]
            at += p
            table[i, :p] = mine.to(torch.int32)
            rows = []
            for x in range(2):
                c = (torch.randn(k, hkv, hd, generator=g) * 2.6).round().clamp(-8, 7)
                b = torch.randint(lo, hi, (k, hkv, hd // 32), generator=g, dtype=torch.uint8)
                w = pack(c)
                for j in range(p):
                    m = min(ps, k - j * ps)
                    codes[mine[j], x, :, :m] = w[j * ps:j * ps + m].transpose(0, 1)
                    scales[mine[j], x, :, :m] = b[j * ps:j * ps + m].transpose(0, 1)
                rows.append((c.double().unflatten(-1, (-1, 32)) * SCALE64[b.long()][..., None]).flatten(-2))
            self.k.append(rows[0])
            self.v.append(rows[1])
        T = sum(n)
        q = torch.randn(T, hq * hd + qpad, generator=g).mul(1.5).to(dtype).to(device)
        self.q = q[:, :hq * hd].unflatten(1, (hq, hd))
        codes, scales = codes.to(device), scales.to(device)
        self.k_cache, self.v_cache, self.k_scales, self.v_scales = codes[:, 0], codes[:, 1], scales[:, 0], scales[:, 1]
        if not interleave:
            self.k_cache, self.v_cache = self.k_cache.contiguous(), self.v_cache.contiguous()
            self.k_scales, self.v_scales = self.k_scales.contiguous(), self.v_scales.contiguous()
        self.table = table.to(device)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=device)
        self.kv = torch.tensor(kv, dtype=torch.int32, device=device)
        self.T, self.max_new = T, max(n + [0])

    def args(self):
        return self.q, self.k_cache, self.v_cache, self.k_scales, self.v_scales, self.table, self.cu, self.kv
