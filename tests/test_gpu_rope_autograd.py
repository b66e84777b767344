"""The rotation next to autograd: outputs that a graph holds, tables that would want a gradient, given positions in the
backward pass, and the kinds of differentiation that the op does not have."""
import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp

pytestmark = pytest.mark.gpu
HQ, HKV, HD, L = 4, 2, 64, 24


def test_k_out_without_k_leaves_q_alone():
    """Refused before anything is launched: a caller who mends the call and tries again rotates q once."""
    q = torch.randn(1, L, HQ, HD, device="cuda")
    before = q.clone()
    with pytest.raises(ValueError, match="k_out"):
        usp.usp_rope(q, None, usp.usp_rope_table(L, HD), q_out=q, k_out=torch.empty(1, L, HKV, HD, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(q, before)
