"""The workspace of usp_paged_attn: one that is sized for the largest step serves the smaller ones, and what an
earlier call or anything else left in it does not reach a result."""
import random

import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from paged_ref import Cache, check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,hd,dt", [(8, 1, 128, torch.bfloat16), (16, 4, 128, torch.bfloat16), (5, 5, 64, torch.bfloat16),
                                          (16, 1, 64, torch.bfloat16), (20, 1, 128, torch.bfloat16),
                                          (64, 1, 64, torch.bfloat16), (8, 2, 64, torch.float32), (6, 1, 128, torch.float32),
                                          (32, 1, 64, torch.float32)])
def test_workspace_of_the_largest_step_serves_every_smaller_one(hq, hkv, hd, dt):
    for most in (2, 4, 7, 33, 300):
        c = Cache([(700, most), (90, 1)], hq, hkv, hd, 16, dt, seed=most)
        q, kc, _, table, _, _ = c.args()
        sizes = [usp.usp_paged_attn_workspace_size(q, kc, table, m) for m in range(most + 1)]
        assert sizes == sorted(sizes)
        ws = torch.empty(sizes[-1], dtype=torch.uint8, device="cuda")
        for m in {1, 2, most // 2, most}:
            out, lse = usp.usp_paged_attn(*c.args(), max_new=m, workspace=ws)
            usp.usp_check()
            check_attention(c, out, lse)


def test_what_is_left_in_the_workspace_reaches_no_result():
    """Calls of every route and many sizes, one after the other in one workspace that starts as NaN bytes: each is
    the definition's, and has the bits that it has in a workspace of zeros."""
    r = random.Random(5)
    kinds = [
        lambda: [(r.randrange(1, 5000), 1) for _ in range(r.randrange(1, 30))],
        lambda: [(r.randrange(300, 3000), r.randrange(1, 300)) for _ in range(r.randrange(1, 4))],
        lambda: [(r.randrange(0, 3000), r.choice([0, 1, 1, 200])) for _ in range(30)],
        lambda: [(r.randrange(0, 60), r.randrange(1, 400)) for _ in range(4)],
        lambda: [(30000, 1), (r.randrange(1, 90), 1)],
    ]
    ws = torch.full((96 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    for n in range(40):
        hkv = r.choice([1, 2, 4])
        c = Cache(kinds[n % 5](), hkv * r.choice([1, 2, 4, 5, 8]), hkv, r.choice([64, 128]), r.choice([16, 64, 256]),
                  torch.float32 if n % 3 == 2 else torch.bfloat16, seed=n)
        zero = usp.usp_paged_attn(*c.args(), max_new=c.max_new, workspace=torch.zeros_like(ws))
        if n % 4 == 0:
            ws.fill_(0xff)
        out, lse = usp.usp_paged_attn(*c.args(), max_new=c.max_new, workspace=ws)
        usp.usp_check()
        check_attention(c, out, lse)
        assert torch.equal(out, zero[0]) and torch.equal(lse, zero[1])
