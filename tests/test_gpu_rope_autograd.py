"""The rotation next to autograd: outputs that a graph holds, tables that would want a gradient, given positions in the
backward pass, and the kinds of differentiation that the op does not have."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import sequence_long_context_zigzag_gb300 as usp
from q4_ref import rope_table, rotate

pytestmark = pytest.mark.gpu
HQ, HKV, HD, L = 4, 2, 64, 24


def leaves(dt=torch.float32):
    return [torch.randn(1, L, h, HD, device="cuda").to(dt).requires_grad_() for h in (HQ, HKV)]


def append_args():
    k = torch.randn(L, HKV, HD, device="cuda")
    kc = torch.zeros(2, HKV, 16, HD, device="cuda")
    return (k, k.clone(), kc, kc.clone(), torch.arange(L, dtype=torch.int32, device="cuda"), usp.usp_rope_table(L, HD)), \
        dict(positions=torch.arange(L, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("leaf", [False, True])
def test_an_output_of_a_graph_is_refused(leaf):
    """The rotation in place of a tensor that autograd follows would leave its gradient unrotated."""
    table = usp.usp_rope_table(L, HD)
    q, k = (x if leaf else x * 2 for x in leaves())
    fresh = [torch.zeros_like(x) for x in (q.detach(), k.detach())]
    before = q.detach().clone(), k.detach().clone()
    for kw in (dict(q_out=q, k_out=k), dict(q_out=q), dict(q_out=fresh[0], k_out=k), dict(q_out=q[:, :, :], k_out=fresh[1])):
        with pytest.raises(ValueError, match="grad"):
            usp.usp_rope(q, k, table, **kw)
    a, kw = append_args()
    with pytest.raises(ValueError, match="grad"):
        usp.usp_rope_append(q[0], *a, **kw, q_out=q[0])
    torch.cuda.synchronize()
    assert torch.equal(q, before[0]) and torch.equal(k, before[1]) and not fresh[0].any() and not a[2].any()
    # where no gradient is recorded, as torch's own operations in place
    want = usp.usp_rope(*before, table)
    with torch.no_grad():
        usp.usp_rope(q, k, table, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_an_output_counts_as_modified():
    """A node that saved a tensor notices that it was rotated in place."""
    table = usp.usp_rope_table(L, HD)
    for call in (lambda x: usp.usp_rope(x, None, table, q_out=x),
                 lambda x: usp.usp_rope(torch.randn(1, L, HQ, HD, device="cuda"), x, table, k_out=x),
                 lambda x: usp.usp_rope_append(x[0], *append_args()[0], **append_args()[1], q_out=x[0])):
        w = torch.randn(1, L, HQ, HD, device="cuda", requires_grad=True)
        x = torch.randn(1, L, HQ, HD, device="cuda")
        y = (w * x).sum()
        at = x._version
        call(x)
        assert x._version > at
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
    a, kw = append_args()
    for call in (lambda: usp.usp_rope_append(None, *a, **kw), lambda: usp.usp_cache_append(*a[:5])):
        at = [t._version for t in a[2:4]]
        call()
        assert all(t._version > v for t, v in zip(a[2:4], at))


def test_outputs_in_inference_mode():
    table = usp.usp_rope_table(L, HD)
    with torch.inference_mode():
        q = torch.randn(1, L, HQ, HD, device="cuda")
        want = usp.usp_rope(q, None, table)[0]
        assert usp.usp_rope(q, None, table, q_out=q)[0] is q and torch.equal(q, want)
        a, kw = append_args()
        usp.usp_rope_append(None, *a, **kw)
    torch.cuda.synchronize()


def test_a_table_that_wants_a_gradient_is_refused():
    """The op has no gradient for its table: it is refused instead of left out."""
    q, k = leaves()
    f = (10000.0 ** (-torch.arange(0, HD, 2, device="cuda") / HD)).requires_grad_()
    angle = torch.arange(L, device="cuda")[:, None] * f
    table = torch.cat([angle.cos(), angle.sin()], 1)
    for x, y in ((q, k), (q.detach(), None)):
        with pytest.raises(ValueError, match="table"):
            usp.UspRopeFunction.apply(x, y, table)
    with torch.no_grad():
        got = usp.UspRopeFunction.apply(q, k, table)
    want = usp.UspRopeFunction.apply(q, k, table.detach())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_k_out_without_k_leaves_q_alone():
    """Refused before anything is launched: a caller who mends the call and tries again rotates q once."""
    q = torch.randn(1, L, HQ, HD, device="cuda")
    before = q.clone()
    with pytest.raises(ValueError, match="k_out"):
        usp.usp_rope(q, None, usp.usp_rope_table(L, HD), q_out=q, k_out=torch.empty(1, L, HKV, HD, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(q, before)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("both", [False, True])   # with cu_seqlens beside the positions, which then count
def test_gradient_at_given_positions(dt, interleaved, both):
    table = rope_table(L + 3, 48)
    g = torch.Generator().manual_seed(2)
    given = torch.randint(-2, L + 6, (1, L), generator=g, dtype=torch.int32)   # some of no row of the table
    pos = torch.where((given < 0) | (given >= L + 3), -1, given).flatten()
    cu = torch.tensor([0, 5, L], dtype=torch.int32, device="cuda") if both else None
    q, k = leaves(dt)
    up = [torch.randn_like(x, requires_grad=True) for x in (q, k)]
    y = usp.UspRopeFunction.apply(q, k, table.cuda(), given.cuda(), cu, interleaved)
    for a, x in zip(y, (q, k)):
        assert torch.equal(a.flatten(0, 1), rotate(x.detach().flatten(0, 1), table, pos, interleaved)[0].to(dt))
    d = torch.autograd.grad(y, (q, k), up, create_graph=True)
    for a, x in zip(d, up):
        assert torch.equal(a.flatten(0, 1), rotate(x.detach().flatten(0, 1), table, pos, interleaved, True)[0].to(dt))
    # and their gradient in turn
    w = [torch.randn_like(x) for x in (q, k)]
    for a, x in zip(torch.autograd.grad(d, up, w), w):
        assert torch.equal(a.flatten(0, 1), rotate(x.flatten(0, 1), table, pos, interleaved)[0].to(dt))


def test_other_kinds_of_differentiation_are_refused():
    """Forward mode and torch.func end in an error, never in a result without its derivative."""
    table = usp.usp_rope_table(L, HD)
    q, k = (x.detach() for x in leaves())
    with fwd.dual_level():
        dual = fwd.make_dual(q, torch.ones_like(q))
        with pytest.raises(RuntimeError):
            usp.UspRopeFunction.apply(dual, k, table)
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda x: usp.UspRopeFunction.apply(x, k, table)[0].sum())(q)
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda x: usp.UspRopeFunction.apply(x, None, table)[0])(torch.stack([q, q]))
