"""The appends into a 4-bit cache: bytes equal to those of the definition (tests/q4_ref.py), at ties, at the scales'
borders and ends, for NaN and infinities."""
import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from q4_ref import SCALE64, pack, quantise, rope_table, rotate, values
from test_gpu_rope import APPENDS, Step, i32

pytestmark = pytest.mark.gpu


def test_the_reference_is_consistent():
    c = torch.randint(-8, 8, (5, 64))
    b = torch.randint(0, 256, (5, 2), dtype=torch.uint8)
    x = values(pack(c), b)
    assert torch.equal(x, c.double() * SCALE64[b.long()].repeat_interleave(32, -1))
    assert torch.equal(x.to(torch.bfloat16).double(), x)      # exact in bf16
    y = torch.randn(300, 128)
    q = values(*quantise(y))
    step = SCALE64[quantise(y)[1].long()].repeat_interleave(32, -1)
    assert ((q - y).abs() <= step / 2).all() and (step / 2 <= y.abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1) * 0.075).all()


def empty_cache(pages, hkv, ps, hd, fill=0x5a):
    return [torch.full((pages, hkv, ps, hd // n), fill, dtype=torch.uint8, device="cuda") for n in (2, 2, 32, 32)]


def store(rows_k, rows_v, dt, hd):
    """Both sides' bytes for rows (n, hd), a row per token and head."""
    n = rows_k.shape[0]
    cache = empty_cache(-(-n // 16), 1, 16, hd)
    usp.usp_cache_append_q4(rows_k[:, None].to(dt).cuda(), rows_v[:, None].to(dt).cuda(), *cache,
                            torch.arange(n, dtype=torch.int32, device="cuda"))
    usp.usp_check()
    return [x.transpose(1, 2).reshape(-1, x.shape[-1])[:n].cpu() for x in cache]


def check(x, dt, hd):
    x = x.to(dt)
    y = x.flip(0)
    got = store(x, y, dt, hd)
    (kc, ks), (vc, vs) = quantise(x), quantise(y)
    for name, a, b in zip(("k", "v", "k scales", "v scales"), got, (kc, vc, ks, vs)):
        assert torch.equal(a, b), name


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_values_of_every_kind(dt, hd):
    g = torch.Generator().manual_seed(hd)
    check(torch.randn(4000, hd, generator=g) * torch.exp(4 * torch.randn(4000, 1, generator=g)), dt, hd)
    # whole and half steps: every element at a tie or beside one
    s = SCALE64[torch.randint(0, 256, (4000, hd // 32), generator=g)].repeat_interleave(32, -1)
    x = (torch.randint(-15, 16, (4000, hd), generator=g).double() / 2 * s).float()
    x[:, ::32] = (7.5 * s[:, ::32]).float()
    check(x, dt, hd)
    if dt == torch.float32:
        check(torch.nextafter(x, torch.zeros_like(x)), dt, hd)
        y = torch.nextafter(x, x * 2)
        check(y, dt, hd)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_scales_at_their_borders(dt):
    """Groups whose largest value is 7.5 s for every s, a step above and a step below; the ends of the range."""
    top = (SCALE64 * 7.5).float()
    rows = []
    for t in (top, torch.nextafter(top, top * 2), torch.nextafter(top, torch.zeros_like(top)), top * 1.01, top * 0.99):
        r = t[:, None] * torch.linspace(-1, 1, 64)[None]
        r[:, 0], r[:, 63] = t, -t
        rows.append(r)
    check(torch.cat(rows), dt, 64)
    r = torch.zeros(40, 64)
    r[0], r[1, 3], r[2], r[3, 40] = 0, 1e-30, -1e-38, 1e-45
    r[4], r[5, 7], r[6, 9] = 3e38, -3e38, 28801.0
    check(r, dt, 64)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_nan_and_infinities(dt):
    x = torch.randn(64, 128, generator=torch.Generator().manual_seed(3))
    x[3, 5], x[4, 60], x[5, 127], x[6] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[7, 0], x[7, 1], x[8, 31], x[8, 30] = float("nan"), float("inf"), float("nan"), 1e30
    check(x, dt, 128)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("new,hq,hkv,hd,ps,rot", APPENDS)
def test_append_with_and_without_the_rotation(new, hq, hkv, hd, ps, rot, interleaved, strided, dt):
    s = Step(new, hq, hkv, hd, ps, dt, seed=len(new) + 1, strided=strided)
    s.ps = ps
    table = rope_table(max(c + n for c, n in zip(s.ctx, new)) + 1, rot)
    for turned in (False, True):
        pos = s.pos if turned else torch.zeros_like(s.pos)
        cache = empty_cache(s.pages, hkv, ps, hd)
        if strided:   # K and V, codes and scales, as parts of wider pages
            wide = torch.full((s.pages, 2, hkv * ps * (hd // 2 + hd // 32) + 32), 0x5a, dtype=torch.uint8, device="cuda")
            n = hkv * ps * hd // 2
            cache = [wide[:, i, a:b].unflatten(1, (hkv, ps, -1)) for a, b in ((0, n), (n, n + hkv * ps * hd // 32)) for i in range(2)]
        want = [x.clone() for x in cache]
        at, page, row = s.stored(pos)
        fk = rotate(s.k, table, pos, interleaved)[0] if turned else s.k.float()
        for i, x in ((0, fk), (1, s.v)):
            codes, scales = quantise(x[at])
            want[i][page, :, row], want[2 + i][page, :, row] = codes, scales
        if turned:
            q = usp.usp_rope_append(s.q, s.k, s.v, *cache[:2], s.slots.cuda(), table.cuda(), s.cu, s.kv, k_scales=cache[2],
                                    v_scales=cache[3], interleaved=interleaved)
            assert torch.equal(q[:s.T], rotate(s.q, table, pos, interleaved)[0].to(dt)[:s.T])
        else:
            usp.usp_cache_append_q4(s.k, s.v, *cache, s.slots.cuda())
        usp.usp_check()
        for a, b in zip(cache, want):
            assert torch.equal(a, b)
        if strided:
            assert (wide[:, :, -32:] == 0x5a).all()


def test_offsets_past_32_bits():
    hkv, ps, hd, num = 8, 256, 128, 33000
    cache = empty_cache(num, hkv, ps, hd, 0)
    assert cache[0].numel() > 2 ** 32
    k, v = (torch.randn(40, hkv, hd, device="cuda").bfloat16() for _ in range(2))
    slots = (num * ps - 1 - 3 * torch.arange(40)).to(torch.int32)
    usp.usp_cache_append_q4(k, v, *cache, slots.cuda())
    usp.usp_check()
    page, row = slots.long() // ps, slots.long() % ps
    for i, x in ((0, k), (1, v)):
        codes, scales = quantise(x)
        assert torch.equal(cache[i][page, :, row], codes) and torch.equal(cache[2 + i][page, :, row], scales)


def test_append_in_a_graph_and_on_a_stream():
    s = Step([3, 20], 4, 2, 64, 16, torch.bfloat16, seed=9)
    table = usp.usp_rope_table(300, 64)
    a, b = empty_cache(s.pages, 2, 16, 64), empty_cache(s.pages, 2, 16, 64)

    def step(c, **kw):
        return usp.usp_rope_append(s.q, s.k, s.v, *c[:2], s.slots.cuda() if kw else slots, table, s.cu, s.kv, k_scales=c[2],
                                   v_scales=c[3], **kw)
    slots = s.slots.cuda()
    side = torch.cuda.Stream()
    step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = step(a)
    s.k.mul_(1.7)
    s.kv.add_(5)
    graph.replay()
    torch.cuda.synchronize()
    q2 = step(b, stream=side)
    side.synchronize()
    assert torch.equal(q[:s.T], q2[:s.T]) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_binding_refuses():
    k = torch.zeros(3, 2, 64, device="cuda")
    c = empty_cache(4, 2, 16, 64)
    slots = i32([0, 1, 2])
    for args in ((k, k, c[0], c[1], c[2], c[3][:3]), (k, k, c[0], c[1][:3], c[2], c[3]), (k, k, c[0].int(), c[1].int(), c[2], c[3]),
                 (k, k, c[0], c[1], c[2].float(), c[3].float()), (k[:, :1], k[:, :1], *c), (k, k[:2], *c)):
        with pytest.raises(ValueError):
            usp.usp_cache_append_q4(*args, slots)
    with pytest.raises(ValueError):
        usp.usp_cache_append_q4(k, k, *c, slots[:2])
    with pytest.raises(TypeError):
        usp.usp_cache_append_q4(k.double(), k.double(), *c, slots)
    with pytest.raises(ValueError, match="k_scales"):
        usp.usp_rope_append(None, k, k, c[0], c[1], slots, usp.usp_rope_table(4, 64), i32([0, 3]), i32([3]))
    with pytest.raises(usp.UspError):     # pages of 8 tokens
        usp.usp_cache_append_q4(k, k, *[x[:, :, :8].contiguous() for x in c], slots)
