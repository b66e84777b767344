"""Query rows that are not finite, over bf16 and fp32 paged caches: they stay alone."""
import math

import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from paged_ref import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hkv,hd", [(4, 2, 64), (16, 1, 128), (32, 1, 128)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_query_rows_that_are_not_finite_stay_alone(dt, hq, hkv, hd, value):
    """NaN, or, where all its scores are -inf, what a row without a key gives. Every other row is what it is without it, to the
    rounding: rows worked on together move their maxima together, which scales weights and sums alike, by powers that are off by
    2^-22 (fp32: four of these), and rounds the weights anew (bf16: 2^-8 each way, and out as well)."""
    c = Cache([(700, 3), (300, 1), (900, 150), (1, 1)], hq, hkv, hd, 32, dt, seed=6)
    want = usp.usp_paged_attn(*c.args(), max_new=c.max_new)
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    for t, h, d in ((1, 0, 5), (3, hq - 1, hd - 1), (40, hq // 2, 0), (c.T - 1, 0, 9)):
        c.q[t, h, d] = value
        bad[t, h] = True
    out, lse = usp.usp_paged_attn(*c.args(), max_new=c.max_new)
    usp.usp_check()
    size = max(v.abs().max().item() for v in c.v)
    assert ((out - want[0])[~bad].abs() <= (2.0 ** -20 if dt == torch.float32 else 3 * 2.0 ** -8) * size).all()
    seen = ~bad & (want[1] != -math.inf)
    assert ((lse - want[1])[seen].abs() <= 2.0 ** -18).all() and torch.equal(lse[~bad & ~seen], want[1][~bad & ~seen])
    for o, x in zip(out[bad], lse[bad]):
        assert (o.isnan().all() and x.isnan()) or not math.isnan(value) and not o.any() and x == -math.inf
