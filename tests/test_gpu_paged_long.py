"""Calls of seconds: a tile of rows that has nothing to do in a unit may wait for the next one as long as that unit takes."""
import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from paged_ref import HALF_STEP

pytestmark = pytest.mark.gpu


def test_a_unit_of_two_tiles_behind_a_long_one_of_one():
    """The first CTA's span holds a unit of one tile of rows over 4 * 10^8 keys, which takes some three seconds, and then one of
    two tiles; the other CTAs have a request of many blocks. (All tables name one page over and over.)"""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    hd, ps, long, short, top = 128, 256, 400_000_000, 1000, 2 ** 31 - 1024
    blocks = -(-sms * (long + 10_000_000) // top)        # of 256 tokens: every span is a little longer than the first unit
    new, kvs = [40, 200, 256 * blocks], [long, short, top]
    k = torch.zeros(1, 1, ps, hd, dtype=torch.bfloat16, device="cuda")
    v = torch.nn.functional.one_hot(torch.arange(ps) % hd, hd).to(torch.bfloat16).cuda().view(1, 1, ps, hd)
    table = torch.zeros(3, -(-top // ps), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 40, 240, 240 + new[2]], dtype=torch.int32, device="cuda")
    q = torch.randn(240 + new[2], 1, hd, device="cuda").to(torch.bfloat16)
    out, lse = usp.usp_paged_attn(q, k, v, table, cu, torch.tensor(kvs, dtype=torch.int32, device="cuda"), max_new=new[2], causal=False)
    usp.usp_check()
    # a column's count is exact in a sum below 2^24, and off by 2^-24 a sum above; out is rounded
    at = 0
    for n, kv in zip(new, kvs):
        want = torch.full((hd,), kv // hd, dtype=torch.float64, device="cuda")
        want[:kv % hd] += 1
        want /= kv
        assert ((out[at:at + n, 0].double() - want).abs() <= want * (HALF_STEP[torch.bfloat16] + 2.0 ** -11)).all()
        assert ((lse[at:at + n].double() - torch.log(torch.tensor(float(kv), dtype=torch.float64))).abs() <= 1e-4).all()
        at += n
