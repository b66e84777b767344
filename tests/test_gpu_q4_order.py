"""The kernels of the rotation and of the 4-bit paged cache may start under the end of the grid before them. Here that
grid is one that lets them start at its very beginning and writes their inputs only some time later."""
import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from q4_ref import Q4Cache
from test_gpu_paged_order import Flat, late_copy  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

CALLS = {
    "decode": ([(700, 1), (90, 1), (3000, 1)], 128, torch.bfloat16),
    "chunk": ([(600, 300), (2000, 170)], 128, torch.bfloat16),
    "one tile of rows": ([(6000, 9), (200, 20), (2000, 5)], 128, torch.bfloat16),
    "both": ([(600, 120), (90, 1), (1500, 1)], 64, torch.bfloat16),
    "f32": ([(600, 120), (90, 1), (1500, 1)], 64, torch.float32),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_attention_after_a_grid_that_lets_it_start_early(late_copy, name):  # noqa: F811
    reqs, hd, dt = CALLS[name]
    c = Q4Cache(reqs, 8, 2, hd, 16, dt, seed=70)
    args = [t.contiguous() for t in c.args()]
    want = usp.usp_paged_attn_q4(*args, max_new=c.max_new)
    flat = Flat(args)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(usp.usp_paged_attn_q4_workspace_size(args[0], args[1], args[5], c.max_new), dtype=torch.uint8, device="cuda")
    for n in range(20):
        # lengths that were there before: the call's own reads of them would give other work
        flat.live.fill_(n % 3)
        out.fill_(float("nan"))
        if n % 2:  # the old values lie in the SMs' first-level caches
            usp.usp_paged_attn_q4(*flat.views, max_new=c.max_new, workspace=ws)
        late_copy(flat.true, flat.live, 20000 + 3000 * n, 8 + 40 * (n % 4))
        usp.usp_paged_attn_q4(*flat.views, max_new=c.max_new, out=out, lse=lse, workspace=ws)
        usp.usp_check()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rotation_and_appends_after_a_grid_that_lets_them_start_early(late_copy, dt):  # noqa: F811
    g = torch.Generator().manual_seed(72)
    lens, hq, hkv, hd, ps, num = [300, 1, 0, 700, 1, 90], 4, 2, 64, 16, 120
    T = sum(lens)
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    kv = torch.tensor([n + 40 * i for i, n in enumerate(lens)], dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(T, h, hd, generator=g).to(dt).cuda() for h in (hq, hkv, hkv))
    slots = torch.randperm(num * ps, generator=g)[:T].to(torch.int32).cuda()
    flat = Flat([q, k, v, slots, usp.usp_rope_table(1200, hd), cu, kv])

    def calls(q, k, v, slots, table, cu, kv, first=lambda: None):
        cache = [torch.zeros(num, hkv, ps, hd, dtype=dt, device="cuda") for _ in range(2)]
        cache4 = [[torch.zeros(num, hkv, ps, hd // n, dtype=torch.uint8, device="cuda") for n in (2, 2, 32, 32)] for _ in range(2)]
        outs = []
        for call in (lambda: usp.usp_rope(q[None], k[None], table, cu_seqlens=cu),
                     lambda: [usp.usp_rope_append(q, k, v, *cache, slots, table, cu, kv)],
                     lambda: [usp.usp_rope_append(q, k, v, *cache4[0][:2], slots, table, cu, kv, k_scales=cache4[0][2], v_scales=cache4[0][3])],
                     lambda: usp.usp_cache_append_q4(k, v, *cache4[1], slots)):
            first()
            outs += call()
        usp.usp_check()
        return (*outs, *cache, *cache4[0])
    want = calls(q, k, v, slots, flat.views[4].copy_(usp.usp_rope_table(1200, hd)), cu, kv)
    for n in range(20):
        def first():
            flat.live.fill_(n % 3)
            late_copy(flat.true, flat.live, 20000 + 3000 * n, 8 + 40 * (n % 4))
        assert all(torch.equal(a, b) for a, b in zip(calls(*flat.views, first=first), want))
