"""The paged cache's kernels may start under the end of the grid before them. Here that grid is one that lets them
start at its very beginning and writes their inputs only some time later."""
import ctypes
import os
import subprocess

import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from paged_ref import Cache
from sequence_long_context_zigzag_gb300 import build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def late_copy(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("late") / "late_grid.so")
    subprocess.run([build._nvcc(), *build.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", so,
                    os.path.join(HERE, "late_grid.cu")], check=True)
    f = ctypes.CDLL(so).late_copy
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_ulonglong, ctypes.c_int, ctypes.c_void_p]

    def call(true, live, ns, grid):
        assert f(true.data_ptr(), live.data_ptr(), live.nbytes, ns, grid, torch.cuda.current_stream().cuda_stream) == 0
    return call


class Flat:
    """Tensors in one buffer, and the same places in another that the late grid fills from it."""

    def __init__(self, tensors):
        sizes = [-(-t.numel() * t.element_size() // 256) * 256 for t in tensors]
        self.true = torch.zeros(sum(sizes), dtype=torch.uint8, device="cuda")
        self.live = torch.zeros_like(self.true)
        at, self.views = 0, []
        for t, n in zip(tensors, sizes):
            for buf, keep in ((self.true, False), (self.live, True)):
                v = buf[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
                if keep:
                    self.views.append(v)
                else:
                    v.copy_(t)
            at += n


CALLS = {
    "decode": ([(700, 1), (90, 1), (3000, 1)], 128, torch.bfloat16),
    "chunk": ([(600, 300), (2000, 170)], 128, torch.bfloat16),
    "both": ([(600, 120), (90, 1), (1500, 1)], 64, torch.bfloat16),
    "f32 decode": ([(700, 1), (90, 1), (3000, 1)], 64, torch.float32),
    "f32 both": ([(600, 120), (90, 1), (1500, 1)], 128, torch.float32),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_attention_after_a_grid_that_lets_it_start_early(late_copy, name):
    reqs, hd, dt = CALLS[name]
    c = Cache(reqs, 8, 2, hd, 16, dt, seed=70)
    want = usp.usp_paged_attn(*[t.contiguous() for t in c.args()], max_new=c.max_new)
    flat = Flat([t.contiguous() for t in c.args()])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for n in range(20):
        # lengths that were there before: the call's own reads of them would give other work
        flat.live.fill_(n % 3)
        out.fill_(float("nan"))
        if n % 2:  # the old values lie in the SMs' first-level caches
            usp.usp_paged_attn(*flat.views, max_new=c.max_new, workspace=ws)
        late_copy(flat.true, flat.live, 20000 + 3000 * n, 8 + 40 * (n % 4))
        usp.usp_paged_attn(*flat.views, max_new=c.max_new, out=out, lse=lse, workspace=ws)
        usp.usp_check()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_plan_and_append_after_a_grid_that_lets_them_start_early(late_copy):
    g = torch.Generator().manual_seed(71)
    ps, nreq, num, tokens, hkv, hd = 16, 300, 4000, 5000, 2, 128
    ctx = torch.randint(0, 100, (nreq,), generator=g, dtype=torch.int32).cuda()
    new = torch.randint(0, 17, (nreq,), generator=g, dtype=torch.int32).cuda()
    free = torch.randperm(num, generator=g).to(torch.int32).cuda()
    head, table = torch.tensor([5], dtype=torch.int32, device="cuda"), torch.zeros(nreq, 9, dtype=torch.int32, device="cuda")
    table[:] = torch.randint(0, num, table.shape, generator=g, dtype=torch.int32).cuda()
    want_table = table.clone()
    want = usp.usp_page_plan(ctx, new, free, head, want_table, ps, num, tokens)
    rows = [torch.randn(tokens, hkv, hd, generator=g).cuda().to(torch.bfloat16) for _ in range(2)]
    slots = torch.randperm(num * ps, generator=g)[:tokens].to(torch.int32).cuda()
    want_cache = [torch.zeros(num, hkv, ps, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache = [torch.zeros_like(x) for x in want_cache]
    usp.usp_cache_append(*rows, *want_cache, slots)
    plan, app = Flat([ctx, new, free, head, table]), Flat([*rows, slots])
    got = [torch.empty_like(x) for x in want]
    names = ("slot_map", "cu_new", "kv_lens", "counts")
    for n in range(20):
        plan.live.fill_(n % 3)
        app.live.fill_(n % 3)
        for x in cache:
            x.zero_()
        late_copy(plan.true, plan.live, 20000 + 3000 * n, 8 + 40 * (n % 4))
        usp.usp_page_plan(*plan.views, ps, num, tokens, **dict(zip(names, got)))
        late_copy(app.true, app.live, 20000 + 3000 * n, 8 + 40 * (n % 4))
        usp.usp_cache_append(*app.views[:2], *cache, app.views[2])
        usp.usp_check()
        assert torch.equal(plan.views[4], want_table) and all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(cache, want_cache))
