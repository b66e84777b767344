"""fp32 queries over a 4-bit cache: q and the weights enter the tensor cores as three bf16 terms each, which hold their 24
bits. Data on which the third term of either shows: few keys, whose scores and weights are known to a few half steps.
And query values that are infinite."""
import math

import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from q4_ref import Q4Cache, pack

pytestmark = pytest.mark.gpu
U = 2.0 ** -24   # half a step of fp32
ONE = 160        # the byte of a scale of 1
HEADS = [(1, 1), (8, 1), (12, 1), (6, 2), (16, 1)]   # units of 8 and of 16 rows


def set_rows(c, i, k, v, kb, vb):
    """Codes and scale bytes of request i's rows (keys, hkv, ..)."""
    n = k.shape[0]
    page, row = c.table[i, torch.arange(n, device="cuda") // c.ps].long(), torch.arange(n, device="cuda") % c.ps
    c.k_cache[page, :, row], c.v_cache[page, :, row] = pack(k).cuda(), pack(v).cuda()
    c.k_scales[page, :, row], c.v_scales[page, :, row] = kb.cuda(), vb.cuda()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("new", [1, 2])
def test_every_bit_of_q_reaches_the_score(hq, hkv, hd, new):
    """One key with one element: lse is scale q k. Request d has element d."""
    c = Q4Cache([(1, new)] * hd, hq, hkv, hd, 16, torch.float32, seed=hq)
    g = torch.Generator().manual_seed(hd)
    code, byte = torch.randint(1, 8, (hd,), generator=g), torch.randint(140, 176, (hd,), generator=g, dtype=torch.uint8)
    for d in range(hd):
        k = torch.zeros(1, hkv, hd)
        k[..., d] = code[d]
        set_rows(c, d, k, k, torch.full((1, hkv, hd // 32), int(byte[d]), dtype=torch.uint8),
                 torch.full((1, hkv, hd // 32), ONE, dtype=torch.uint8))
    out, lse = usp.usp_paged_attn_q4(*c.args(), max_new=new, causal=False, scale=0.7)
    usp.usp_check()
    kd = code.double() * (8 + (byte & 7)).double() * 2.0 ** ((byte >> 3).double() - 23)
    d = torch.arange(hd).repeat_interleave(new)
    want = 0.7 * c.q.double().cpu()[torch.arange(hd * new), :, d] * kd[d][:, None]
    # half steps: the score's sum, scale log2(e) and its two factors (3), the maximum, m + log2(l), ln 2 and the product with it;
    # l = 1 to 2 units in the last place of exp2f, and log2f's 2 at 1: 2^-21
    bound = 9 * U * want.abs() + 2.0 ** -21
    err = (lse.double().cpu() - want).abs()
    assert (err <= bound).all(), f"{(err / bound).max().item():.3g} bounds"
    # (two terms of q, off by 2^-17 on average, would be far outside)
    assert (2.0 ** -17 * want.abs() > 2 * bound).float().mean() > 0.5
    # out: weight 1, value k. The product of a weight of 24 bits and a value of 7 is cut to 24 (2 half steps), 1 / l and the
    # product with it are rounded
    v = torch.nn.functional.one_hot(d, hd)[:, None] * code[d][:, None, None].double()
    assert ((out.double().cpu() - v).abs() <= 4 * U * v).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("kv", [16, 60])
def test_every_bit_of_the_weights_reaches_out(hq, hkv, hd, kv):
    """Small scores of single-element keys, V one-hot by key: out is the weights. 16 keys are one warp's, 60 two warps'."""
    n = 40
    c = Q4Cache([(kv, 1)] * n, hq, hkv, hd, 16, torch.float32, seed=kv)
    g = torch.Generator().manual_seed(hd)
    codes, bytes_ = torch.randint(1, 8, (n, kv), generator=g), torch.randint(128, 136, (n, kv), generator=g, dtype=torch.uint8)
    at = torch.arange(kv)
    for i in range(n):
        k, v = torch.zeros(kv, hkv, hd), torch.zeros(kv, hkv, hd)
        k[at, :, (at * 5 + i) % hd] = codes[i][:, None].float()
        v[at, :, at] = 1
        set_rows(c, i, k, v, bytes_[i][:, None, None].expand(-1, hkv, hd // 32), torch.full((kv, hkv, hd // 32), ONE, dtype=torch.uint8))
    out, _ = usp.usp_paged_attn_q4(*c.args(), max_new=1, scale=0.35)
    usp.usp_check()
    kd = codes.double() * (8 + (bytes_ & 7)).double() * 2.0 ** ((bytes_ >> 3).double() - 23)     # (n, kv)
    dim = (at[None] * 5 + torch.arange(n)[:, None]) % hd
    s = 0.35 * c.q.double().cpu().gather(2, dim[:, None].expand(-1, hq, -1)) * kd[:, None]
    want = s.softmax(-1)
    # relative, half steps: a weight and the normaliser each by its scores (the sum, scale log2(e) and its factors, the maximum,
    # the argument: 6 of the largest score) and exp2f (4: 2 units in the last place); the sums of l (a dozen), 1 / l and the
    # product (2). Warps that join add an ex2 each to a weight and to the normaliser, of 2^-22 (4).
    e = 2 * (6 * s.abs().amax(-1, keepdim=True) + 4) + 14 + (8 if kv > 32 else 0)
    err = (out.double().cpu()[..., :kv] - want).abs() / want
    assert (err <= e * U).all(), f"{(err / (e * U)).max().item():.3g} bounds"
    # (the third terms of such weights are 2^-16 of them at most, and many of them more than the bound)
    assert (e * U).median() < 2.0 ** -18
    assert not out[..., kv:].any()


@pytest.mark.parametrize("hq,hkv,hd", [(4, 2, 64), (8, 1, 128), (16, 1, 64), (12, 1, 128), (20, 1, 128)])
@pytest.mark.parametrize("reqs", [[(3000, 1), (700, 2), (40000, 1)], [(1500, 37), (900, 9)]], ids=["tokens", "chunks"])
def test_error_of_fp32_queries(reqs, hq, hkv, hd):
    """Out against 64 bits, relative, over all elements together. The errors of different keys are independent and add up as
    the weighted values do, so it is that of a weight: exp2f (2^-22 at most), the score's sum, its scale and the argument
    (half steps of numbers of a few units), some 3e-7 at these scores; what all keys share, the sums and 1 / l, is a few half steps
    more. Two bf16 terms of q or of the weights instead of three give 3e-6 and more."""
    c = Q4Cache(reqs, hq, hkv, hd, 64, torch.float32, seed=5)
    c.q.mul_(0.5)
    out, _ = usp.usp_paged_attn_q4(*c.args(), max_new=c.max_new)
    usp.usp_check()
    t = 0
    for i, (kv, n) in enumerate(reqs):
        k, v = (x[i].cuda().repeat_interleave(hq // hkv, 1) for x in (c.k, c.v))
        s = torch.einsum("qhd,khd->hqk", c.q[t:t + n].double(), k) / math.sqrt(hd)
        s = s.masked_fill(torch.arange(kv, device="cuda") > kv - n + torch.arange(n, device="cuda")[:, None], -math.inf)
        want = torch.einsum("hqk,khd->qhd", s.softmax(-1), v)
        err = (out[t:t + n].double() - want).norm() / want.norm()
        assert err <= 2.0 ** -21, f"request {i}: {err.item():.3g}"
        t += n


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hkv,hd", [(4, 2, 64), (16, 1, 128), (32, 1, 128)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_query_rows_that_are_not_finite_stay_alone(dt, hq, hkv, hd, value):
    """A row with an infinite or NaN value has no finite score: NaN, or, where all its scores are -inf, what a row without a key
    gives. Every other row is what it is without it."""
    c = Q4Cache([(700, 3), (300, 1), (900, 150), (1, 1)], hq, hkv, hd, 32, dt, seed=6)
    want = usp.usp_paged_attn_q4(*c.args(), max_new=c.max_new)
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    for t, h, d in ((1, 0, 5), (3, hq - 1, hd - 1), (40, hq // 2, 0), (c.T - 1, 0, 9)):
        c.q[t, h, d] = value
        bad[t, h] = True
    out, lse = usp.usp_paged_attn_q4(*c.args(), max_new=c.max_new)
    usp.usp_check()
    assert torch.equal(out[~bad], want[0][~bad]) and torch.equal(lse[~bad], want[1][~bad])
    for o, x in zip(out[bad], lse[bad]):
        assert (o.isnan().all() and x.isnan()) or (value < 0 or value > 0) and not o.any() and x == -math.inf
