"""The rotation of whole sequences and its gradient, and the append with the rotation on the way, against the formula
in 64 bits with bounds from the roundings the kernels make (tests/q4_ref.py)."""
import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from q4_ref import rope_table, rotate

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def near(got, want, bound):
    err = (got.double() - want).abs()
    assert not torch.isnan(err).any()
    assert (err <= bound).all(), f"off by up to {(err / bound).max().item():.3g} bounds"


def test_table_holds_the_angles_cosines_and_sines():
    t = usp.usp_rope_table(300, 64, base=500.0)
    assert t.dtype == torch.float32 and t.is_cuda
    near(t.cpu(), rope_table(300, 64, 500.0).double(), 2.0 ** -24 + 1e-12)
    f = torch.tensor([1.0, 0.3, 1e-3], dtype=torch.float64)
    t = usp.usp_rope_table(200000, 6, inv_freq=f)
    a = 199999 * f
    near(t[-1].cpu(), torch.cat([a.cos(), a.sin()]), 2.0 ** -24 + 1e-9)


ROPES = [(1, 1, 1, 1, 64, 64), (1, 77, 4, 2, 128, 128), (3, 50, 5, 1, 64, 32), (2, 333, 8, 8, 128, 48), (1, 2000, 32, 8, 128, 128),
         (2, 64, 1, 0, 64, 16), (1, 129, 40, 3, 128, 112), (4, 1, 2, 2, 64, 48)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bs,L,hq,hkv,hd,rot", ROPES)
def test_rope_matches_the_formula(bs, L, hq, hkv, hd, rot, interleaved, dt):
    g = torch.Generator().manual_seed(L)
    table = rope_table(L + 3, rot)
    q = torch.randn(bs, L, hq, hd, generator=g).to(dt).cuda()
    k = torch.randn(bs, L, hkv, hd, generator=g).to(dt).cuda() if hkv else None
    cut = sorted(torch.randint(0, L + 1, (3,), generator=g).tolist())
    cu = [0] + cut + [L]                             # an empty sample may be among them
    given = torch.randint(-2, L + 6, (bs, L), generator=g, dtype=torch.int32)  # some of no row of the table
    packed = torch.cat([torch.arange(b - a) for a, b in zip(cu[:-1], cu[1:])])
    for kw, pos in (({}, torch.arange(L).repeat(bs)), (dict(cu_seqlens=i32(cu)), packed.repeat(bs)),
                    (dict(positions=given.cuda()), torch.where((given < 0) | (given >= L + 3), -1, given).flatten())):
        for inverse in (False, True):
            got = usp.usp_rope(q, k, table.cuda(), interleaved=interleaved, inverse=inverse, **kw)
            usp.usp_check()
            for x, y in zip((q, k), got):
                if x is None:
                    assert y is None
                    continue
                f, want, bound = rotate(x.flatten(0, 1), table, pos, interleaved, inverse)
                near(y.flatten(0, 1), want, bound)
                assert torch.equal(y.flatten(0, 1), f.to(dt))     # every operation rounded on its own
                assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rope_strides_in_place_and_streams(dt):
    """q and k as slices of a fused projection, rotated in place: the rest of it keeps its bytes."""
    bs, L, hq, hkv, hd = 2, 70, 6, 2, 64
    table = usp.usp_rope_table(L, hd)
    all_ = torch.randn(bs, L, hq + 2 * hkv, hd, device="cuda").to(dt)
    q, k, v = all_[:, :, :hq], all_[:, :, hq:hq + hkv], all_[:, :, hq + hkv:].clone()
    want = usp.usp_rope(q, k, table)
    alone = usp.usp_rope(q.contiguous(), k.contiguous(), table)
    assert all(torch.equal(a, b) for a, b in zip(want, alone))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = usp.usp_rope(q, k, table, q_out=q, k_out=k, stream=s)
    s.synchronize()
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(all_[:, :, hq + hkv:], v)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved, dt):
    """Against the formula's gradient, and (fp32) against differences: the op is linear, so a difference over any step is
    its derivative."""
    bs, L, hq, hkv, hd, rot = 2, 45, 4, 2, 64, 48
    table, cu = usp.usp_rope_table(L, rot), i32([0, 13, 13, 45])
    pos = torch.cat([torch.arange(13), torch.arange(32)]).repeat(bs)
    q, k = (torch.randn(bs, L, h, hd, device="cuda").to(dt).requires_grad_() for h in (hq, hkv))
    gq, gk = (torch.randn(bs, L, h, hd, device="cuda").to(dt) for h in (hq, hkv))
    yq, yk = usp.UspRopeFunction.apply(q, k, table, None, cu, interleaved)
    dq, dk = torch.autograd.grad((yq, yk), (q, k), (gq, gk))
    for d, up in ((dq, gq), (dk, gk)):
        _, want, bound = rotate(up.flatten(0, 1), table.cpu(), pos, interleaved, True)
        near(d.flatten(0, 1), want, bound)
    if dt == torch.float32:
        with torch.no_grad():
            step = torch.randn_like(q)
            z = usp.usp_rope(q + step, k, table, cu_seqlens=cu, interleaved=interleaved)[0]
            lhs, rhs = ((z - yq).double() * gq).sum(), (dq.double() * step).sum()
            # each of the two sums' terms is off by a few half steps of values of a few units
            assert abs(lhs - rhs) <= 8 * 2.0 ** -24 * ((z.abs() + yq.abs()).double() * gq.abs()).sum()
    # only one of the outputs used; no k at all
    assert torch.equal(torch.autograd.grad(usp.UspRopeFunction.apply(q, k, table, None, cu, interleaved)[0], q, gq)[0], dq)
    y, none = usp.UspRopeFunction.apply(q, None, table, None, cu, interleaved)
    assert none is None and torch.equal(torch.autograd.grad(y, q, gq)[0], dq)


def test_rope_second_gradient():
    """The gradient is differentiable in turn: of <rotate back(g), u> with respect to g it is the rotation of u."""
    table, cu = usp.usp_rope_table(30, 64), i32([0, 11, 30])
    q, k = (torch.randn(1, 30, h, 64, device="cuda", requires_grad=True) for h in (3, 2))
    gq, gk = (torch.randn_like(x, requires_grad=True) for x in (q, k))
    uq, uk = torch.randn_like(q), torch.randn_like(k)
    dq, dk = torch.autograd.grad(usp.UspRopeFunction.apply(q, k, table, None, cu, True), (q, k), (gq, gk), create_graph=True)
    second = torch.autograd.grad((dq, dk), (gq, gk), (uq, uk))
    want = usp.usp_rope(uq, uk, table, cu_seqlens=cu, interleaved=True)
    assert all(torch.equal(a, b) for a, b in zip(second, want))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rope_gradients_that_lie_anywhere(dt):
    """Gradients that come expanded, and as parts of a tensor that start at no 16-byte boundary."""
    table = usp.usp_rope_table(9, 64)
    q, k = (torch.randn(2, 9, h, 64, device="cuda").to(dt).requires_grad_() for h in (3, 1))
    yq, yk = usp.UspRopeFunction.apply(q, k, table)
    one = torch.ones_like
    want = usp.usp_rope(one(q), one(k), table, inverse=True)
    got = torch.autograd.grad(yq.sum() + yk.sum(), (q, k), retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    up = torch.randn(1 + q.numel() + k.numel(), device="cuda").to(dt)
    got = torch.autograd.grad(torch.cat([up.new_zeros(1), yq.flatten(), yk.flatten()]), (q, k), up)
    want = usp.usp_rope(up[1:q.numel() + 1].clone().view_as(q), up[q.numel() + 1:].clone().view_as(k), table, inverse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rope_gradients_in_a_graph():
    """Forward and backward through the op, captured and replayed on other values; strided leaves."""
    table = usp.usp_rope_table(24, 128)
    base = torch.randn(2, 24, 8, 128, device="cuda").bfloat16()
    both = base.clone().requires_grad_()
    gq, gk = (torch.randn(2, 24, h, 128, device="cuda").bfloat16() for h in (5, 3))

    def step():
        y = usp.UspRopeFunction.apply(both[:, :, :5], both[:, :, 5:], table)
        return (*y, torch.autograd.grad(y, both, (gq, gk))[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        both.copy_(base.flip(0))
        gq.neg_()
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    pos = torch.arange(24).repeat(2)
    for d, up in ((want[2][:, :, :5], gq), (want[2][:, :, 5:], gk)):
        _, w, bound = rotate(up.flatten(0, 1), table.cpu(), pos, False, True)
        near(d.flatten(0, 1), w, bound)


def test_rotated_attention_step():
    """Rotation and attention as a training step uses them: forward and gradients of the two ops together agree with
    the formula's, differentiated by torch in 64 bits."""
    bs, L, hq, hkv, hd = 1, 96, 4, 2, 64
    g = torch.Generator().manual_seed(3)
    x = [torch.randn(bs, L, h, hd, generator=g).cuda() for h in (hq, hkv, hkv)]
    table = usp.usp_rope_table(L, hd)
    leaves = [t.clone().requires_grad_() for t in x]
    q, k = usp.UspRopeFunction.apply(leaves[0], leaves[1], table)
    out = usp.UspAttentionFunction.apply(q, k, leaves[2], 2, 2)
    up = torch.randn(out.shape, generator=g).cuda()
    grads = torch.autograd.grad(out, leaves, up)
    usp.usp_check()
    ref = [t.double().requires_grad_() for t in x]
    c, s = table[:, None, :hd // 2].double(), table[:, None, hd // 2:].double()

    def rot(t):
        u, v = t[..., :hd // 2], t[..., hd // 2:]
        return torch.cat([u * c - v * s, v * c + u * s], -1)
    rq, rk = rot(ref[0]), rot(ref[1]).repeat_interleave(hq // hkv, 2)
    e = torch.einsum("blhd,bmhd->bhlm", rq, rk) / hd ** 0.5
    e = e.masked_fill(torch.ones(L, L, device="cuda", dtype=torch.bool).triu(1), -torch.inf)
    o = torch.einsum("bhlm,bmhd->blhd", e.softmax(-1), ref[2].repeat_interleave(hq // hkv, 2))
    want = torch.autograd.grad(o, ref, up.double())
    # fp32 throughout: sums of some hundred terms of a few units, a few dozen half steps
    near(out, o.detach(), 2e-5)
    for a, b in zip(grads, want):
        near(a, b, 2e-4)


def test_rope_in_a_graph_and_beside_it():
    """Captured and replayed on other values, forward and backward."""
    L, table = 40, usp.usp_rope_table(40, 64)
    q, k = (torch.randn(1, L, h, 64, device="cuda", requires_grad=True) for h in (4, 2))
    gq, gk = torch.randn_like(q), torch.randn_like(k)

    def step():
        with torch.no_grad():
            y = usp.usp_rope(q, k, table)
            return (*y, *usp.usp_rope(gq, gk, table, inverse=True))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(2):
        with torch.no_grad():
            for t in (q, k, gq, gk):
                t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


# ---- append with the rotation ------------------------------------------------------------------------------------
APPENDS = [([1], 4, 1, 64, 16, 64), ([1] * 70, 8, 2, 128, 64, 128), ([5, 0, 300, 1, 77], 5, 1, 64, 32, 48),
           ([700, 0, 0, 1], 32, 8, 128, 16, 128), ([3], 16, 1, 128, 256, 112), ([1, 2] * 800, 2, 2, 64, 16, 32)]


class Step:
    """One step's q, k, v with slots and lengths, padded by `pad` tokens of no request."""

    def __init__(self, new, hq, hkv, hd, ps, dt, seed, pad=3, strided=False):
        g = torch.Generator().manual_seed(seed)
        nreq, T = len(new), sum(new)
        self.ctx = torch.randint(0, 90, (nreq,), generator=g).tolist()
        self.pos = torch.cat([torch.arange(c, c + n) for c, n in zip(self.ctx, new)] + [torch.full((pad,), -1)])
        self.pages = -(-(T + pad) // ps) + 4
        slots = torch.randperm(self.pages * ps, generator=g)[:T + pad].to(torch.int32)
        slots[torch.rand(T + pad, generator=g) < 0.1] = -1
        if T > 4:
            slots[1], slots[2] = self.pages * ps, 2 ** 31 - 1
        self.T, self.pad, self.slots = T, pad, slots
        row = (hq + 2 * hkv) * hd
        wide = torch.randn(T + pad, row + (16 if strided else 0), generator=g).to(dt).cuda()
        parts = wide[:, :hq * hd], wide[:, hq * hd:(hq + hkv) * hd], wide[:, (hq + hkv) * hd:row]
        self.q, self.k, self.v = [x.unflatten(1, (-1, hd)) if strided else x.contiguous().unflatten(1, (-1, hd)) for x in parts]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        self.cu, self.kv = i32(cu), i32([c + n for c, n in zip(self.ctx, new)])

    def stored(self, pos):
        """Tokens that are stored, with their pages and rows."""
        s = self.slots.long()
        at = torch.nonzero((s >= 0) & (s < self.pages * self.ps) & (pos >= 0))[:, 0]
        return at, s[at] // self.ps, s[at] % self.ps


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("new,hq,hkv,hd,ps,rot", APPENDS)
def test_rope_append(new, hq, hkv, hd, ps, rot, interleaved, strided, dt):
    s = Step(new, hq, hkv, hd, ps, dt, seed=len(new), strided=strided)
    s.ps = ps
    table = rope_table(max(c + n for c, n in zip(s.ctx, new)) + 1, rot)
    buf = torch.randn(s.pages, 2, hkv, ps, hd, device="cuda").to(dt)
    g = torch.Generator().manual_seed(1)
    given = torch.randint(-1, table.shape[0] + 2, (s.T + s.pad,), generator=g, dtype=torch.int32)
    for kw, pos in ((dict(cu_new=s.cu, kv_lens=s.kv), s.pos),
                    (dict(positions=given.cuda()), torch.where(given >= table.shape[0], -1, given).long())):
        kc, vc = buf[:, 0].clone(), buf[:, 1].clone()
        if strided:
            b = buf.clone()
            kc, vc = b[:, 0], b[:, 1]
        want_k, want_v, q_out = kc.clone(), vc.clone(), torch.full((s.T + s.pad, hq, hd), 7.0, device="cuda").to(dt)
        fk, fq = (rotate(x, table, pos, interleaved)[0].to(dt) for x in (s.k, s.q))
        at, page, row = s.stored(pos)
        want_k[page, :, row], want_v[page, :, row] = fk[at], s.v[at]
        got = usp.usp_rope_append(s.q, s.k, s.v, kc, vc, s.slots.cuda(), table.cuda(), interleaved=interleaved, q_out=q_out, **kw)
        usp.usp_check()
        assert got is q_out
        assert torch.equal(q_out[pos >= 0], fq[pos >= 0]) and (q_out[pos < 0] == 7).all()
        assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    # no q: the caches alone
    kc, vc = buf[:, 0].clone(), buf[:, 1].clone()
    assert usp.usp_rope_append(None, s.k, s.v, kc, vc, s.slots.cuda(), table.cuda(), positions=given.cuda(), interleaved=interleaved) is None
    usp.usp_check()
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_rope_append_in_place_and_without_requests():
    s = Step([4, 9], 4, 2, 64, 16, torch.bfloat16, seed=5, pad=0)
    table = usp.usp_rope_table(200, 64)
    kc, vc = (torch.zeros(s.pages, 2, 16, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    want = usp.usp_rope_append(s.q, s.k, s.v, kc, vc, s.slots.cuda(), table, s.cu, s.kv)
    q = s.q.clone()
    assert usp.usp_rope_append(q, s.k, s.v, kc, vc, s.slots.cuda(), table, s.cu, s.kv, q_out=q) is q
    assert torch.equal(q, want)
    before = kc.clone()
    usp.usp_rope_append(q, s.k, s.v, kc, vc, s.slots.cuda(), table, s.cu[:1], s.kv[:0], q_out=q)  # no request: no position
    usp.usp_rope_append(q[:0], s.k[:0], s.v[:0], kc, vc, s.slots[:0].cuda(), table, s.cu[:1], s.kv[:0])
    usp.usp_check()
    assert torch.equal(q, want) and torch.equal(kc, before)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rope_append_offsets_past_32_bits(dt):
    """A cache of more than 2^31 elements: the last pages."""
    hkv, ps, hd, num = 8, 256, 128, 8300
    kc, vc = (torch.empty(num, hkv, ps, hd, dtype=dt, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    k, v, q = (torch.randn(40, h, hd, device="cuda").to(dt) for h in (hkv, hkv, 2))
    table = rope_table(50, hd)
    pos = torch.arange(40)
    slots = (num * ps - 1 - 3 * pos).to(torch.int32)
    usp.usp_rope_append(q, k, v, kc, vc, slots.cuda(), table.cuda(), positions=pos.to(torch.int32).cuda())
    usp.usp_check()
    page, row = slots.long() // ps, slots.long() % ps
    assert torch.equal(kc[page, :, row], rotate(k, table, pos, False)[0].to(dt)) and torch.equal(vc[page, :, row], v)


def test_binding_refuses():
    q, k = torch.zeros(1, 8, 4, 64, device="cuda"), torch.zeros(1, 8, 2, 64, device="cuda")
    t = usp.usp_rope_table(8, 64)
    for bad in (dict(q_out=torch.zeros(1, 8, 4, 128, device="cuda")), dict(positions=torch.zeros(7, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(8, dtype=torch.int32)), dict(cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            usp.usp_rope(q, k, t, **bad)
    for args in ((q, k[:, :7], t), (q, k, t.double()), (q, k.bfloat16(), t), (q.transpose(1, 2), k, t), (q, k, t.cpu())):
        with pytest.raises(ValueError):
            usp.usp_rope(*args)
    for args in ((q, k, t[:7]), (q, k, usp.usp_rope_table(8, 24)), (q, k, usp.usp_rope_table(8, 128))):
        with pytest.raises(usp.UspError):
            usp.usp_rope(*args)
    with pytest.raises(ValueError):
        usp.usp_rope(q, None, t, k_out=torch.empty_like(k))
    kc = torch.zeros(4, 2, 16, 64, device="cuda")
    slots, cu, kv = i32([0] * 8), i32([0, 8]), i32([8])
    q, k = q[0], k[0]
    for args in ((q, k, k, kc, kc, slots, t, cu, cu), (q, k, k, kc, kc, slots[:7], t, cu, kv), (q[:7], k, k, kc, kc, slots, t, cu, kv),
                 (q, k, k, kc.bfloat16(), kc.bfloat16(), slots, t, cu, kv), (q, q, q, kc, kc, slots, t, cu, kv)):
        with pytest.raises(ValueError):
            usp.usp_rope_append(*args)
    with pytest.raises(TypeError):
        usp.usp_rope_append(q, k, k, kc, kc, slots, t)
    with pytest.raises(usp.UspError):  # no table: nothing to rotate by
        usp.usp_rope_append(None, k, k, kc, kc, slots, None, cu, kv)
