"""The workspace of usp_paged_attn: one that is sized for the largest step serves the smaller ones."""
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
