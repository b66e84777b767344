"""Sums over a million keys in one CTA: the tensor cores cut what they add up to fp32 towards zero, which must not gather."""
import math

import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from q4_ref import SCALE64, values

pytestmark = pytest.mark.gpu
KV, HKV, PS = 2 ** 20, 4, 256


def long_values(hd, bytes_):
    """V of one sign and odd scales, columns of different means: (codes, scale bytes, means in 64 bits)."""
    g = torch.Generator(device="cuda").manual_seed(hd)
    n = KV // PS
    v = torch.empty(n, HKV, PS, hd // 2, dtype=torch.uint8, device="cuda")
    b = torch.randint(*bytes_, (n, HKV, PS, hd // 32), generator=g, dtype=torch.uint8, device="cuda")
    mean = torch.empty(HKV, hd, dtype=torch.float64, device="cuda")
    s = SCALE64.cuda()[b.long()]
    top = torch.linspace(1.2, 7.99, hd, device="cuda")    # codes 1 .. top of a column
    perm = torch.randperm(hd, generator=g, device="cuda")
    for h in range(HKV):
        c = (1 + torch.rand(n, PS, hd, generator=g, device="cuda") * (top[perm] - 1)).to(torch.uint8)
        mean[h] = (c.double() * s[:, h].repeat_interleave(32, -1)).sum((0, 1)) / KV
        c = c.unflatten(-1, (-1, 8))[..., [0, 2, 4, 6, 1, 3, 5, 7]].flatten(-2)   # nibble n of a word: value 2 n, or 2 (n - 4) + 1
        v[:, h] = c[..., 0::2] | c[..., 1::2] << 4
    return v, b, mean


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G", [4, 8, 12, 24, 32])
@pytest.mark.parametrize("bytes_", [(140, 152), (100, 152)], ids=["alike", "spread"])   # spread: values of more bits
def test_sums_of_a_million_keys(G, hd, bytes_):
    """K = 0: every weight is 1 and out the mean of V, rounded to bf16. Beside that rounding: a product cuts its sum by less than
    2^-22 of it, at most 1024 products follow one another, on a sum that grows from 0 (2^-13); 32 to 128 such sums, of four
    warps, and 1 / l are rounded (2^-16)."""
    v, b, mean = long_values(hd, bytes_)
    nreq = 160                                      # more units than CTAs: most hold one whole
    k = torch.zeros_like(v)
    table = torch.arange(KV // PS, dtype=torch.int32, device="cuda").expand(nreq, -1).contiguous()
    cu = torch.arange(nreq + 1, dtype=torch.int32, device="cuda")
    q = torch.randn(nreq, HKV * G, hd, device="cuda").to(torch.bfloat16)
    out, lse = usp.usp_paged_attn_q4(q, k, v, b, b, table, cu, torch.full_like(cu[1:], KV), max_new=1)
    usp.usp_check()
    want = mean.repeat_interleave(G, 0)
    half = 2.0 ** (want.log2().floor() - 8)
    err = (out.double() - want).abs()
    assert (err <= half + (2.0 ** -13 + 2.0 ** -16) * want).all(), f"off by {((err - half) / want).max().item():.2g} beside the rounding"
    assert ((lse.double() - math.log(KV)).abs() <= 1e-5).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G,new", [(1, 1), (5, 1), (16, 1), (7, 3), (32, 1)])
def test_scores_that_grow_and_fall(G, new, hd):
    """Scores of a ramp over the keys, up or down by the head, so that the maximum moves through all of a long unit or lies at its
    beginning; some rows have none (a request with fewer keys than new tokens). Weights are rounded to bf16 (2^-8 of sum p |v| at
    most) and so is out; scores are off by hd 2^-24 scale sum |q k|, below 2^-10."""
    kv, nreq = 100000, 128
    n = -(-kv // PS)
    g = torch.Generator(device="cuda").manual_seed(G + hd)
    byte = lambda lo, hi, last: torch.randint(lo, hi, (n, HKV, PS, last), generator=g, dtype=torch.uint8, device="cuda")
    k, v, ks, vs = byte(0, 256, hd // 2), byte(0, 256, hd // 2), byte(128, 140, hd // 32), byte(140, 152, hd // 32)
    ramp = torch.linspace(-8, 7.99, n * PS, device="cuda").floor().long().view(n, 1, PS).expand(-1, HKV, -1)
    k[..., 0] = ((ramp & 15) | (k[..., 0] & 0xf0)).to(torch.uint8)      # value 0 of a row (nibble 0 of its first word)
    ks[..., 0] = 152                                                    # 8 2^-4 = 0.5
    table = torch.arange(n, dtype=torch.int32, device="cuda").expand(nreq, -1).contiguous()
    cu = torch.arange(nreq + 1, dtype=torch.int32, device="cuda") * new
    kvs = torch.full_like(cu[1:], kv)
    kvs[-1] = new - 1
    one = torch.randn(new, HKV * G, hd, generator=g, device="cuda") * 0.3
    one[..., 0] = torch.where(torch.arange(HKV * G, device="cuda") % 2 == 0, 1.0, -1.0) * 5 * hd ** 0.5
    q = one.to(torch.bfloat16).repeat(nreq, 1, 1)
    out, lse = usp.usp_paged_attn_q4(q, k, v, ks, vs, table, cu, kvs, max_new=new)
    usp.usp_check()
    o, s_ = out.unflatten(0, (nreq, new)), lse.unflatten(0, (nreq, new))
    assert (o[:-1] == o[:1]).float().mean() > 0.9   # the same request over and over, cut elsewhere
    for h in range(HKV):
        K, V = (values(c[:, h], s[:, h]).flatten(0, 1)[:kv] for c, s in ((k, ks), (v, vs)))
        e = torch.einsum("qgd,kd->qgk", one.to(torch.bfloat16)[:, h * G:(h + 1) * G].double(), K) / hd ** 0.5
        for m, rows in ((kv, slice(0, nreq - 1)), (new - 1, slice(nreq - 1, nreq))):
            x = e[..., :m].masked_fill(torch.arange(m, device="cuda") > m - new + torch.arange(new, device="cuda")[:, None, None], -math.inf)
            w = x.softmax(-1).nan_to_num(0.0)
            want, size, l = w @ V[:m], w @ V[:m].abs(), x.logsumexp(-1) if m else torch.full(x.shape[:2], -math.inf, device="cuda")
            got, gl = o[rows, :, h * G:(h + 1) * G].double(), s_[rows, :, h * G:(h + 1) * G].double()
            assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * size).all()
            assert torch.equal(gl.isinf(), l.isinf().expand_as(gl))
            assert ((gl - l).nan_to_num(0.0).abs() <= 2.0 ** -10).all()


# ---- the kernels of many rows: pieces of 65536 keys --------------------------------------------------------------


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G,new,nreq", [(4, 9, 100), (4, 32, 60), (4, 64, 50), (8, 64, 25), (40, 1, 100)])
@pytest.mark.parametrize("q4", [True, False])
def test_sums_of_a_million_keys_of_many_rows(G, new, nreq, hd, q4):
    """As above, over a 4-bit and over a bf16 cache; 4096 products follow one another at most (2^-11)."""
    table = torch.arange(KV // PS, dtype=torch.int32, device="cuda").expand(nreq, -1).contiguous()
    cu = torch.arange(nreq + 1, dtype=torch.int32, device="cuda") * new
    q = torch.randn(nreq * new, HKV * G, hd, device="cuda").to(torch.bfloat16)
    rest = (table, cu, torch.full_like(cu[1:], KV))
    if q4:
        v, b, mean = long_values(hd, (100, 152))
        out, lse = usp.usp_paged_attn_q4(q, torch.zeros_like(v), v, b, b, *rest, max_new=new, causal=False)
    else:
        v = (torch.rand(KV // PS, HKV, PS, hd, device="cuda") + torch.linspace(0.3, 2.0, hd, device="cuda")).to(torch.bfloat16)
        mean = v.double().sum((0, 2)) / KV
        out, lse = usp.usp_paged_attn(q, torch.zeros_like(v), v, *rest, max_new=new, causal=False)
    usp.usp_check()
    want = mean.repeat_interleave(G, 0)
    half = 2.0 ** (want.log2().floor() - 8)
    err = (out.double() - want).abs()
    assert (err <= half + (2.0 ** -11 + 2.0 ** -16) * want).all(), f"off by {((err - half) / want).max().item():.2g} beside the rounding"
    assert ((lse.double() - math.log(KV)).abs() <= 1e-5).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kv", [65556, 140000])    # (20 keys in the second piece, of which a unit's first tile of rows sees none)
@pytest.mark.parametrize("G,new", [(4, 9), (4, 64), (8, 40), (40, 1), (1, 300)])
@pytest.mark.parametrize("q4", [True, False])
def test_scores_that_grow_and_fall_of_many_rows(G, new, kv, hd, q4):
    """As above."""
    nreq, n = 128 if new < 100 else 60, -(-kv // PS)
    g = torch.Generator(device="cuda").manual_seed(G + hd)
    ramp = torch.linspace(-8, 7.99, n * PS, device="cuda").floor().view(n, 1, PS).expand(-1, HKV, -1)
    if q4:
        byte = lambda lo, hi, last: torch.randint(lo, hi, (n, HKV, PS, last), generator=g, dtype=torch.uint8, device="cuda")
        k, v, ks, vs = byte(0, 256, hd // 2), byte(0, 256, hd // 2), byte(128, 140, hd // 32), byte(140, 152, hd // 32)
        k[..., 0] = ((ramp.long() & 15) | (k[..., 0] & 0xf0)).to(torch.uint8)
        ks[..., 0] = 152
        cache, K_, V_ = (k, v, ks, vs), values(k, ks), values(v, vs)
    else:
        k, v = (torch.randn(n, HKV, PS, hd, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        k[..., 0] = ramp / 2
        cache, K_, V_ = (k, v), k.double(), v.double()
    table = torch.arange(n, dtype=torch.int32, device="cuda").expand(nreq, -1).contiguous()
    cu = torch.arange(nreq + 1, dtype=torch.int32, device="cuda") * new
    kvs = torch.full_like(cu[1:], kv)
    kvs[-1] = new - 1
    one = torch.randn(new, HKV * G, hd, generator=g, device="cuda") * 0.3
    one[..., 0] = torch.where(torch.arange(HKV * G, device="cuda") % 2 == 0, 1.0, -1.0) * 5 * hd ** 0.5
    one = one.to(torch.bfloat16)
    call = usp.usp_paged_attn_q4 if q4 else usp.usp_paged_attn
    out, lse = call(one.repeat(nreq, 1, 1), *cache, table, cu, kvs, max_new=new)
    usp.usp_check()
    out, lse = out.unflatten(0, (nreq, new)), lse.unflatten(0, (nreq, new))
    for h in range(HKV):
        K, V = (x[:, h].flatten(0, 1)[:kv] for x in (K_, V_))
        e = torch.einsum("qgd,kd->qgk", one[:, h * G:(h + 1) * G].double(), K) / hd ** 0.5
        for m, rows in ((kv, slice(0, nreq - 1)), (new - 1, slice(nreq - 1, nreq))):
            x = e[..., :m].masked_fill(torch.arange(m, device="cuda") > m - new + torch.arange(new, device="cuda")[:, None, None], -math.inf)
            w = x.softmax(-1).nan_to_num(0.0)
            want, size, l = w @ V[:m], w @ V[:m].abs(), x.logsumexp(-1) if m else torch.full(x.shape[:2], -math.inf, device="cuda")
            got, gl = out[rows, :, h * G:(h + 1) * G].double(), lse[rows, :, h * G:(h + 1) * G].double()
            assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * size).all()
            assert torch.equal(gl.isinf(), l.isinf().expand_as(gl))
            assert ((gl - l).nan_to_num(0.0).abs() <= 2.0 ** -10).all()
