"""Attention over a 4-bit paged cache, against the definition in 64 bits over what the cache's bytes stand for, with
bounds derived from the roundings the kernels make (tests/paged_ref.py: the same as over a bf16 or fp32 cache, whose values
these are; fp32: the three bf16 terms of a value hold its 24 bits)."""
import random

import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from paged_ref import attention64, check_attention
from q4_ref import Q4Cache, quantise, rope_table, rotate, values

pytestmark = pytest.mark.gpu

DECODE = [(1, 1), (17, 1), (64, 1), (65, 1), (0, 0), (300, 1), (0, 1), (1000, 1), (5, 0), (128, 1), (129, 1), (255, 1)]
CHUNKS = [(1, 1), (130, 130), (129, 2), (300, 257), (0, 0), (700, 64), (65, 65), (1000, 1), (400, 33)]
SHORT = [(3, 40), (0, 7), (200, 300), (1, 2)]   # fewer keys than new tokens: the first rows see nothing


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attend(c, **kw):
    # poisoned outputs: every row of a request has to be written
    kw.setdefault("out", torch.full_like(c.q.contiguous(), float("nan")))
    kw.setdefault("lse", torch.full(c.q.shape[:2], float("nan"), device="cuda"))
    r = usp.usp_paged_attn_q4(*c.args(), **kw)
    usp.usp_check()
    return r


@pytest.mark.parametrize("reqs", [DECODE, CHUNKS, SHORT, [(4000, 1)], [(3001, 500)], [(257, 257)], [(700, 5), (90, 3)]],
                         ids=["decode", "chunks", "short", "one-decode", "one-chunk", "one-prompt", "few"])
@pytest.mark.parametrize("hq,hkv,hd,ps,dt", [
    (8, 2, 128, 16, torch.bfloat16), (4, 4, 64, 64, torch.bfloat16), (8, 1, 128, 128, torch.bfloat16),
    (10, 2, 64, 32, torch.bfloat16), (7, 1, 128, 256, torch.bfloat16), (32, 1, 64, 16, torch.bfloat16),
    (128, 1, 128, 64, torch.bfloat16), (24, 2, 128, 32, torch.bfloat16), (4, 2, 64, 16, torch.float32),
    (3, 1, 128, 256, torch.float32), (16, 1, 64, 32, torch.float32), (128, 1, 128, 16, torch.float32)])
def test_attention_matches_definition(reqs, hq, hkv, hd, ps, dt):
    c = Q4Cache(reqs, hq, hkv, hd, ps, dt, seed=hq + hd)
    # (also without the host's bound, and with one that is too small: the same definition)
    for m in (c.max_new, None, 1):
        out, lse = attend(c, max_new=m)
        check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hd", [64, 128])
def test_scales_of_many_sizes(hd, dt):
    c = Q4Cache([(900, 1), (333, 40), (500, 300)], 8, 2, hd, 16, dt, seed=2, wide=True)
    for m in (c.max_new, 1):
        out, lse = attend(c, max_new=m)
        check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("reqs", [DECODE, CHUNKS, SHORT], ids=["decode", "chunks", "short"])
def test_without_the_causal_mask(reqs, dt):
    c = Q4Cache(reqs, 8, 2, 64, 32, dt, seed=1)
    out, lse = attend(c, causal=False, scale=0.3)
    check_attention(c, out, lse, causal=False, scale=0.3)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("reqs", [DECODE, CHUNKS], ids=["decode", "chunks"])
def test_strides_and_foreign_rows(reqs, dt):
    """q and out as slices of wider rows, interleaved caches, a wider table; rows of no request and the columns beside
    out keep their bytes."""
    c = Q4Cache(reqs, 8, 2, 128, 16, dt, seed=2, interleave=True, qpad=64)
    T, hq, hd = c.q.shape
    wide = torch.full((T + 9, hq * hd + 32), 7.0, dtype=dt, device="cuda")
    q = torch.full((T + 9, hq * hd + 64), float("nan"), dtype=dt, device="cuda")
    q[4:4 + T, :hq * hd] = c.q.flatten(1)
    lse = torch.full((T + 9, hq), 7.0, device="cuda")
    table = torch.full((c.table.shape[0], c.table.shape[1] + 5), 2 ** 30, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    out = wide[:, :hq * hd].unflatten(1, (hq, hd))
    usp.usp_paged_attn_q4(q[:, :hq * hd].unflatten(1, (hq, hd)), *c.args()[1:5], table[:, :c.table.shape[1]], c.cu + 4, c.kv,
                          out=out, lse=lse)
    usp.usp_check()
    check_attention(c, out[4:4 + T], lse[4:4 + T])
    assert (wide[:4] == 7).all() and (wide[4 + T:] == 7).all() and (wide[:, hq * hd:] == 7).all()
    assert (lse[:4] == 7).all() and (lse[4 + T:] == 7).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [1, 150])
def test_pages_outside_the_cache_read_as_zeros(dt, new):
    c = Q4Cache([(600, new), (90, 1)], 4, 2, 64, 32, dt, seed=3)
    for col, page in {1: -1, 4: c.k_cache.shape[0], 6: 2 ** 31 - 1, 7: -2 ** 31}.items():
        c.table[0, col] = page
        c.k[0][col * 32:(col + 1) * 32] = 0
        c.v[0][col * 32:(col + 1) * 32] = 0
    out, lse = attend(c)
    check_attention(c, out, lse)
    c.kv[1] = 2 ** 31 - 1                      # more keys than the table has room for
    c.table[1] = c.table[0]
    c.table[1, -1] = 0
    out, lse = attend(c)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_many_requests(dt):
    r = random.Random(4)
    reqs = [(k, min(k, r.choice([0, 1, 1, 1, 2, 30]))) for k in (r.choice([0, 1, 16, 33, 90]) for _ in range(2500))]
    c = Q4Cache(reqs, 4, 2, 64, 16, dt, seed=4)
    out, lse = attend(c)
    check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_peaked_and_large_scores(dt):
    c = Q4Cache([(900, 1), (500, 200), (64, 64)], 8, 2, 128, 64, dt, seed=5)
    c.q.mul_(24)
    out, lse = attend(c)
    check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hkv,hd", [(8, 1, 128), (5, 1, 64), (6, 2, 64)])
@pytest.mark.parametrize("reqs", [[(60000, 1)], [(30, 1), (25000, 1), (27000, 2), (7, 0), (100, 1)], [(25000, 37), (300, 1)]],
                         ids=["one", "some", "chunk"])
def test_units_of_many_parts(reqs, hq, hkv, hd, dt):
    c = Q4Cache(reqs, hq, hkv, hd, 64, dt, seed=10)
    out, lse = attend(c, max_new=c.max_new)
    check_attention(c, out, lse)


@pytest.mark.parametrize("hq,hkv,hd", [(8, 8, 64), (16, 4, 128), (24, 3, 64), (128, 1, 128), (12, 4, 128)])
def test_long_prompts(hq, hkv, hd):
    """Several units of 256 rows for each SM; rows of no request and columns beside out stay as they were."""
    T = 160 * 2 * 256 * hkv // hq // hkv + 700
    c = Q4Cache([(T, T), (333, 129), (65, 65)], hq, hkv, hd, 128, torch.bfloat16, seed=11)
    wide = torch.full((c.T + 5, hq * hd + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :hq * hd].unflatten(1, (hq, hd))
    lse = torch.full((c.T + 5, hq), 7.0, device="cuda")
    q = torch.cat([c.q.contiguous(), c.q[:5]])
    usp.usp_paged_attn_q4(q, *c.args()[1:], out=out, lse=lse)
    usp.usp_check()
    assert (wide[:, hq * hd:] == 7).all() and (wide[c.T:] == 7).all() and (lse[c.T:] == 7).all()
    # the long request in the definition's memory: its last rows, and its first
    n = 300
    tail, head = Q4Cache.__new__(Q4Cache), Q4Cache.__new__(Q4Cache)
    tail.__dict__.update(c.__dict__)
    tail.reqs, tail.q, tail.T = [(T, n), (333, 129), (65, 65)], c.q[T - n:], c.T - T + n
    check_attention(tail, out[T - n:c.T], lse[T - n:c.T])
    head.__dict__.update(c.__dict__)
    head.reqs, head.q, head.T, head.k, head.v = [(n, n)], c.q[:n], n, [c.k[0][:n]], [c.v[0][:n]]
    check_attention(head, out[:n], lse[:n])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("reqs", [[(200, 2000)], [(300, 40)] + [(0, 40)] * 30 + [(300, 40)], [(0, 90)] * 9,
                                  [(1, 500), (900, 40), (2, 700), (0, 50), (40, 1)]],
                         ids=["one-request", "between", "only", "mixed"])
def test_runs_of_units_without_a_key(reqs, dt):
    c = Q4Cache(reqs, 8, 2, 64, 32, dt, seed=9)
    for kw in (dict(max_new=c.max_new), dict(max_new=1), dict(max_new=c.max_new, causal=False)):
        out, lse = attend(c, **kw)
        check_attention(c, out, lse, causal=kw.get("causal", True))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("reqs", [[(500, 1), (64, 1), (9000, 1)], [(300, 150), (2000, 70), (80, 80)]], ids=["decode", "chunks"])
def test_a_nan_query_row_is_nan_and_stays_alone(reqs, dt):
    c = Q4Cache(reqs, 8, 2, 64, 32, dt, seed=8)
    q = c.q.clone()
    want = [x.clone() for x in attend(c)]
    hit = torch.zeros(c.T, c.hq, dtype=torch.bool, device="cuda")
    for t, h in [(0, 3), (c.T // 2, 6), (c.T - 1, 0)]:
        c.q[t, h, 5] = float("nan")
        hit[t, h] = True
    out, lse = attend(c)
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    out[hit], lse[hit], c.q = want[0][hit], want[1][hit], q
    check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_very_large_or_small_query(dt):
    """Rows of q far from 1: the scores' scale makes up for them."""
    for f in (1e30, 1e-30):
        c = Q4Cache([(300, 1), (200, 90)], 8, 2, 64, 32, dt, seed=12)
        c.q = (c.q.float() * f).to(dt)
        out, lse = attend(c, scale=0.125 / f)
        check_attention(c, out, lse, scale=0.125 / f)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hd,ps", [(128, 64), (64, 16), (128, 16), (64, 256)])
@pytest.mark.parametrize("hq,hkv,most", [(12, 1, 1), (10, 2, 3), (8, 2, 5), (8, 1, 3), (24, 1, 1), (8, 2, 8), (31, 1, 1), (6, 2, 10)])
def test_units_of_nine_to_thirty_two_rows(hq, hkv, most, hd, ps, causal):
    """Two to four tiles of 8 rows, the last one in part: units cut between CTAs, without a key, with fewer keys than new
    tokens; also where a request has more new tokens than the host says."""
    reqs = [(26000, most), (200, most), (15, 1), (129, max(1, most - 1)), (0, most), (128, most), (1, most), (31000, 1), (7, 0)]
    c = Q4Cache(reqs + [(450 + 130 * i, most) for i in range(6)], hq, hkv, hd, ps, torch.bfloat16, seed=81, wide=True)
    out, lse = attend(c, max_new=c.max_new, causal=causal)
    check_attention(c, out, lse, causal)
    again = attend(c, max_new=c.max_new, causal=causal)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    c = Q4Cache([(300, 40), (5000, most)], hq, hkv, hd, ps, torch.bfloat16, seed=82)
    out, lse = attend(c, max_new=most, causal=causal)
    check_attention(c, out, lse, causal)


def test_a_nan_query_row_among_twenty(hd=128):
    c = Q4Cache([(900, 5), (64, 5), (20000, 5)], 8, 2, hd, 64, torch.bfloat16, seed=83)
    c.q[7, 3] = float("nan")
    out, lse = attend(c, max_new=5)
    assert torch.isnan(out[7, 3]).all() and torch.isnan(lse[7, 3])
    c.q[7, 3] = 0
    out2, lse2 = attend(c, max_new=5)
    keep = torch.ones(c.T, 8, dtype=torch.bool, device="cuda")
    keep[7, 3] = False
    assert torch.equal(out[keep], out2[keep]) and torch.equal(lse[keep], lse2[keep])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,hd,ps", [(8, 2, 128, 64), (8, 1, 64, 16), (5, 1, 128, 128), (40, 1, 64, 32)])
@pytest.mark.parametrize("reqs", [
    [(30000, 9)], [(26000, 12), (200, 6), (15, 12), (129, 5), (0, 5), (128, 11), (1, 7), (31000, 10)],
    [(500 + 130 * i, 5 + i) for i in range(12)], [(6, 12), (300, 12), (2, 9)]], ids=["one", "mixed", "twelve", "few keys"])
def test_units_of_one_tile_of_rows(reqs, hq, hkv, hd, ps, causal):
    """More rows than the kernel for few takes, and no more than a tile: the key tiles go to two states, which are joined;
    odd numbers of tiles, one tile, none, units cut between CTAs; rows without a key in either."""
    c = Q4Cache(reqs, hq, hkv, hd, ps, torch.bfloat16, seed=80, wide=True)
    out, lse = attend(c, max_new=c.max_new, causal=causal)
    check_attention(c, out, lse, causal)
    again = attend(c, max_new=c.max_new, causal=causal)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_same_bits_on_every_run(dt):
    c = Q4Cache([(5000, 1), (3000, 300), (40, 40), (2500, 1)], 8, 2, 128, 16, dt, seed=6)
    a = [x.clone() for x in attend(c)]
    for _ in range(3):
        b = attend(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_on_another_stream_and_in_a_graph():
    c = Q4Cache([(700, 1), (90, 1), (1300, 1)], 8, 2, 128, 16, torch.bfloat16, seed=7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = usp.usp_paged_attn_q4(*c.args(), max_new=1, stream=s)
    s.synchronize()
    check_attention(c, out, lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go, gl = usp.usp_paged_attn_q4(*c.args(), max_new=1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(go, out) and torch.equal(gl, lse)
    c.kv.copy_(i32([650, 1, 1300]))
    for i, kv in enumerate((650, 1, 1300)):
        c.reqs[i] = (kv, 1)
        c.k[i], c.v[i] = c.k[i][:kv], c.v[i][:kv]
    g.replay()
    torch.cuda.synchronize()
    check_attention(c, go, gl)


@pytest.mark.parametrize("hq,hkv,hd,ps,dt", [(8, 2, 128, 64, torch.bfloat16), (4, 4, 64, 16, torch.float32)])
def test_rotated_prompt_chunks_and_tokens_through_the_cache(hq, hkv, hd, ps, dt):
    """A serving loop: prompts in chunks, then token by token; plan, rotated append into the 4-bit cache, attention each
    step. The caches end with the definition's bytes, and every step agrees with the definition over them."""
    g = torch.Generator().manual_seed(8)
    L, nreq, num = [520, 300], 2, 64
    r = [[torch.randn(n, h, hd, generator=g).to(dt).cuda() for h in (hq, hkv, hkv)] for n in L]
    kc, vc = (torch.randint(0, 256, (num, hkv, ps, hd // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.randint(0, 256, (num, hkv, ps, hd // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.full((nreq, 40), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(num, generator=g).to(torch.int32).cuda()
    head, ctx, rope = i32([0]), i32([0, 0]), rope_table(600, hd)
    outs, lses, at = [[], []], [[], []], [0, 0]
    for new in [[257, 100], [200, 0], [60, 199]] + [[1, 1]] + [[1, 0]] * 2:
        T = sum(new)
        q, k, v = [torch.cat([r[i][x][at[i]:at[i] + new[i]] for i in range(nreq)]) for x in range(3)]
        slots, cu, kv, counts = usp.usp_page_plan(ctx, i32(new), free, head, table, ps, num, T)
        q = usp.usp_rope_append(q, k, v, kc, vc, slots, rope.cuda(), cu, kv, k_scales=ks, v_scales=vs)
        o, z = usp.usp_paged_attn_q4(q, kc, vc, ks, vs, table, cu, kv, max(new))
        usp.usp_check()
        assert counts.tolist()[0] == T and counts.tolist()[2] == 0
        t = 0
        for i in range(nreq):
            outs[i].append(o[t:t + new[i]])
            lses[i].append(z[t:t + new[i]])
            at[i] += new[i]
            t += new[i]
        ctx, head = kv, counts[1:2]
    assert at == L

    class Whole:
        reqs, T = [(n, n) for n in L], sum(L)
    Whole.hq, Whole.hkv, Whole.hd, Whole.dtype = hq, hkv, hd, dt
    Whole.q, Whole.k, Whole.v = [], [], []
    for i, n in enumerate(L):
        pos = torch.arange(n)
        Whole.q.append(rotate(r[i][0], rope, pos, False)[0].to(dt))
        kb, vb = quantise(rotate(r[i][1], rope, pos, False)[0]), quantise(r[i][2])
        page, row = table[i, pos.cuda() // ps].long(), (pos % ps).cuda()
        for cache, want in ((kc, kb[0]), (ks, kb[1]), (vc, vb[0]), (vs, vb[1])):
            assert torch.equal(cache[page, :, row], want)
        Whole.k.append(values(*kb))
        Whole.v.append(values(*vb))
    Whole.q = torch.cat(Whole.q)
    out, lse = torch.cat(outs[0] + outs[1]), torch.cat(lses[0] + lses[1])
    check_attention(Whole, out, lse)
    # and it stays near the attention over what was appended: a quarter of a step of noise on every key and value
    Whole.k, Whole.v = [rotate(x[1], rope, torch.arange(len(x[1])), False)[1] for x in r], [x[2].double() for x in r]
    full, _, _, _ = attention64(Whole)
    assert ((out.double() - full).norm() / full.norm()) < 0.25


def test_parts_of_a_sequence_merge():
    """Two halves of the keys: the partials merge (usp_lse_merge) to the whole."""
    c = Q4Cache([(1000, 1), (640, 1)], 8, 2, 128, 64, torch.float32, seed=9)
    parts = []
    for lo, hi in ((0, 320), (320, None)):
        kv = i32([len(c.k[i][lo:hi]) for i in range(2)])
        table = c.table[:, lo // 64:].contiguous() if lo else c.table
        parts.append(usp.usp_paged_attn_q4(c.q, *c.args()[1:5], table, c.cu, kv, 1, causal=False))
    usp.usp_lse_merge(parts[0][0], parts[0][1], parts[1][0], parts[1][1])
    usp.usp_check()
    o, z = parts[0]
    ref, lref, bo, bl = attention64(c, causal=False)
    assert ((o.double() - ref).abs() <= 3 * bo + 2.0 ** -20 * ref.abs()).all()
    assert ((z.double() - lref).abs() <= 3 * bl + 2.0 ** -20).all()


def test_fewer_tokens_than_a_tile_of_queries():
    for new, hq, hkv, hd in ((9, 8, 2, 128), (17, 2, 2, 64), (33, 1, 1, 128), (3, 64, 2, 64)):
        c = Q4Cache([(new + 60, new)], hq, hkv, hd, 16, torch.bfloat16, seed=new)
        out, lse = attend(c, max_new=new)
        check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_shared_pages(dt):
    c = Q4Cache([(300, 1), (290, 40), (256, 1)], 8, 2, 64, 64, dt, seed=21)
    for i in (1, 2):
        c.table[i, :4] = c.table[0, :4]
        c.k[i][:256], c.v[i][:256] = c.k[0][:256], c.v[0][:256]
    out, lse = attend(c)
    check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [1, 70])
def test_offsets_past_32_bits(dt, new):
    """A cache of more than 2^32 bytes of codes: append to and attend over its last pages."""
    hkv, ps, hd, num = 8, 256, 128, 32768 - 8
    c = Q4Cache([(600, new), (256, new)], 16, hkv, hd, ps, dt, seed=22)
    cache = [torch.empty(num, hkv, ps, hd // n, dtype=torch.uint8, device="cuda") for n in (2, 2, 32, 32)]
    assert cache[0].numel() > 2 ** 32 - 2 ** 24 and cache[0].numel() + cache[1].numel() > 2 ** 32
    pages = [[num - 1, num - 5, num - 3], [num - 2]]
    c.table = i32([pages[0], pages[1] + [-1, -1]])
    slots = i32([pages[i][p // ps] * ps + p % ps for i, (n, _) in enumerate(c.reqs) for p in range(n)])
    k, v = torch.cat(c.k).float().cuda(), torch.cat(c.v).float().cuda()
    usp.usp_cache_append_q4(k, v, *cache, slots)
    c.k = list(values(*quantise(k.cpu())).split([600, 256]))
    c.v = list(values(*quantise(v.cpu())).split([600, 256]))
    c.k_cache, c.v_cache, c.k_scales, c.v_scales = cache
    out, lse = attend(c)
    check_attention(c, out, lse)


def test_calls_on_three_streams_keep_their_bits():
    r = random.Random(1)

    def make(i):
        reqs = [[(r.randrange(1, 4000), 1) for _ in range(r.randrange(1, 40))],
                [(r.randrange(300, 3000), r.randrange(1, 300)) for _ in range(r.randrange(1, 5))],
                [(r.randrange(100, 2500),) * 2 for _ in range(r.randrange(1, 4))],
                [(r.randrange(200, 3000), r.choice([1, 1, 1, 200])) for _ in range(20)]][i % 4]
        hkv = r.choice([1, 2, 4])
        c = Q4Cache(reqs, hkv * r.choice([1, 2, 4, 5, 8]), hkv, r.choice([64, 128]), r.choice([16, 64, 256]),
                    torch.float32 if i % 5 == 4 else torch.bfloat16, seed=i)
        return c, [x.clone() for x in attend(c, max_new=c.max_new)]
    calls, streams = [make(i) for i in range(20)], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(200):
        wrong = []
        for _ in range(40):
            c, want = r.choice(calls)
            with torch.cuda.stream(r.choice(streams)):
                out, lse = torch.full_like(want[0], float("nan")), torch.full_like(want[1], float("nan"))
                usp.usp_paged_attn_q4(*c.args(), max_new=c.max_new, out=out, lse=lse)
                wrong.append((out != want[0]).sum() + (lse != want[1]).sum())
        torch.cuda.synchronize()
        assert sum(int(x) for x in wrong) == 0
    usp.usp_check()


def test_short_chunks_on_three_streams_keep_their_bits():
    """As above, units of 9 to 128 rows: several tiles of 8 rows with one state, and one tile of 128 with two."""
    r = random.Random(2)

    def make(i):
        G, rows = r.choice([1, 2, 4, 5, 8, 12, 16]), [16, 24, 32, 100][i % 4]
        most = max(1, rows // G)
        reqs = [(r.randrange(most, 6000), r.randrange(max(1, most - 1), most + 1)) for _ in range(r.randrange(1, 20))]
        hkv = r.choice([1, 2, 4])
        c = Q4Cache(reqs, hkv * G, hkv, r.choice([64, 128]), r.choice([16, 64, 256]), torch.bfloat16, seed=100 + i)
        return c, [x.clone() for x in attend(c, max_new=most)], most
    calls, streams = [make(i) for i in range(20)], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(200):
        wrong = []
        for _ in range(40):
            c, want, most = r.choice(calls)
            with torch.cuda.stream(r.choice(streams)):
                out, lse = torch.full_like(want[0], float("nan")), torch.full_like(want[1], float("nan"))
                usp.usp_paged_attn_q4(*c.args(), max_new=most, out=out, lse=lse)
                wrong.append((out != want[0]).sum() + (lse != want[1]).sum())
        torch.cuda.synchronize()
        assert sum(int(x) for x in wrong) == 0
    usp.usp_check()


@pytest.mark.parametrize("hq,hkv,hd,dt", [(8, 1, 128, torch.bfloat16), (16, 4, 128, torch.bfloat16), (5, 5, 64, torch.bfloat16),
                                          (20, 1, 128, torch.bfloat16), (64, 1, 64, torch.bfloat16), (8, 2, 64, torch.float32),
                                          (32, 1, 128, torch.float32)])
def test_workspace_of_the_largest_step_serves_every_smaller_one(hq, hkv, hd, dt):
    for most in (2, 4, 7, 33, 300):
        c = Q4Cache([(700, most), (90, 1)], hq, hkv, hd, 16, dt, seed=most)
        sizes = [usp.usp_paged_attn_q4_workspace_size(c.q, c.k_cache, c.table, m) for m in range(most + 1)]
        assert sizes == sorted(sizes)
        ws = torch.full((sizes[-1],), 0xff, dtype=torch.uint8, device="cuda")
        for m in {1, 2, most // 2, most}:
            out, lse = attend(c, max_new=m, workspace=ws)
            check_attention(c, out, lse)


def test_what_is_left_in_the_workspace_reaches_no_result():
    r = random.Random(5)
    kinds = [
        lambda: [(r.randrange(1, 5000), 1) for _ in range(r.randrange(1, 30))],
        lambda: [(r.randrange(300, 3000), r.randrange(1, 300)) for _ in range(r.randrange(1, 4))],
        lambda: [(r.randrange(0, 3000), r.choice([0, 1, 1, 200])) for _ in range(30)],
        lambda: [(r.randrange(0, 60), r.randrange(1, 400)) for _ in range(4)],
        lambda: [(30000, 1), (r.randrange(1, 90), 1)],
    ]
    ws = torch.full((96 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    for n in range(30):
        hkv = r.choice([1, 2, 4])
        c = Q4Cache(kinds[n % 5](), hkv * r.choice([1, 2, 4, 5, 8]), hkv, r.choice([64, 128]), r.choice([16, 64, 256]),
                    torch.float32 if n % 3 == 2 else torch.bfloat16, seed=n)
        zero = attend(c, max_new=c.max_new, workspace=torch.zeros_like(ws))
        if n % 4 == 0:
            ws.fill_(0xff)
        out, lse = attend(c, max_new=c.max_new, workspace=ws)
        check_attention(c, out, lse)
        assert torch.equal(out, zero[0]) and torch.equal(lse, zero[1])


def test_whole_step_in_one_graph():
    """Plan, rotated append and attention captured together and replayed for other lengths, with -1 slots behind the
    last token."""
    hq, hkv, hd, ps, num, cap = 8, 2, 64, 16, 80, 64
    g = torch.Generator().manual_seed(40)
    cache = [torch.zeros(num, hkv, ps, hd // n, dtype=torch.uint8, device="cuda") for n in (2, 2, 32, 32)]
    table, free = torch.full((2, 30), -1, dtype=torch.int32, device="cuda"), torch.arange(num, dtype=torch.int32, device="cuda")
    ctx, new, head, rope = i32([0, 0]), i32([0, 0]), i32([0]), rope_table(500, hd)
    rope_d = rope.cuda()
    q, k, v = (torch.zeros(cap, h, hd, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))

    def step():
        slots, cu, kv, counts = usp.usp_page_plan(ctx, new, free, head, table, ps, num, cap)
        y = usp.usp_rope_append(q, k, v, *cache[:2], slots, rope_d, cu, kv, k_scales=cache[2], v_scales=cache[3])
        return (*usp.usp_paged_attn_q4(y, *cache, table, cu, kv), kv, counts)
    step()
    usp.usp_check()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, kv, counts = step()

    class C:
        k, v, dtype = [torch.empty(0, hkv, hd).double()] * 2, [torch.empty(0, hkv, hd).double()] * 2, torch.bfloat16
    C.hq, C.hkv, C.hd = hq, hkv, hd
    for lens in ([40, 13], [1, 1], [0, 50], [30, 0]):
        T = sum(lens)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).to(t.dtype))
        new.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        at, rows = 0, []
        for i, n in enumerate(lens):
            pos = len(C.k[i]) + torch.arange(n)
            rows.append(rotate(q[at:at + n].cpu(), rope, pos, False)[0].to(q.dtype))
            C.k[i] = torch.cat([C.k[i], values(*quantise(rotate(k[at:at + n].cpu(), rope, pos, False)[0]))])
            C.v[i] = torch.cat([C.v[i], values(*quantise(v[at:at + n].cpu()))])
            at += n
        C.reqs, C.T, C.q = [(len(C.k[i]), lens[i]) for i in range(2)], T, torch.cat(rows).cuda()
        check_attention(C, out[:T], lse[:T])
        assert counts.tolist()[0] == T and counts.tolist()[2] == 0
        ctx.copy_(kv)
        head.copy_(counts[1:2])


def test_no_work_after_a_recorded_timeout_until_it_is_checked():
    from sequence_long_context_zigzag_gb300 import _abi
    c = Q4Cache([(500, 1), (300, 80)], 8, 2, 128, 16, torch.bfloat16, seed=50)
    _abi.check("usp_selftest_timeout", _abi.load().usp_selftest_timeout(1000, torch.cuda.current_stream().cuda_stream))
    with pytest.raises(usp.UspError) as e:
        attend(c)
    assert e.value.status == _abi.USP_ERR_TIMEOUT
    out, lse = attend(c)
    check_attention(c, out, lse)


def test_binding_refuses():
    c = Q4Cache([(50, 2), (20, 1)], 4, 2, 64, 16, torch.bfloat16)
    q, kc, vc, ks, vs, table, cu, kv = c.args()
    for bad in (dict(lse=torch.empty(3, 5, device="cuda")), dict(out=torch.empty(3, 4, 128, device="cuda")),
                dict(workspace=torch.empty(10, dtype=torch.uint8)), dict(lse=torch.empty(c.T, 4))):
        with pytest.raises(ValueError):
            usp.usp_paged_attn_q4(*c.args(), **bad)
    for args in ((q, kc.int(), vc.int(), ks, vs, table, cu, kv), (q, kc, vc, ks[:, :, :8], vs[:, :, :8], table, cu, kv),
                 (q, kc, vc, ks, vs, table.cpu(), cu, kv), (q, kc, vc, ks, vs, table[:1], cu, kv), (q, kc, vc, ks, vs, table, cu[:2], kv),
                 (torch.zeros(3, 4, 128, device="cuda"), kc, vc, ks, vs, table, cu, kv), (q, kc, vc[:2], ks, vs, table, cu, kv)):
        with pytest.raises(ValueError):
            usp.usp_paged_attn_q4(*args)
    with pytest.raises(TypeError):
        usp.usp_paged_attn_q4(q.half(), kc, vc, ks, vs, table, cu, kv)
    with pytest.raises(usp.UspError):
        usp.usp_paged_attn_q4(*c.args(), max_new=-1)
    with pytest.raises(usp.UspError):
        usp.usp_paged_attn_q4(*c.args(), workspace=torch.empty(128, dtype=torch.uint8, device="cuda"))
    with pytest.raises(usp.UspError):   # pages of 8 tokens
        usp.usp_paged_attn_q4(q, *[x[:, :, :8].contiguous() for x in (kc, vc, ks, vs)], table, cu, kv)
    n = usp.usp_paged_attn_q4_workspace_size(q, kc, table, 2)
    out, lse = usp.usp_paged_attn_q4(*c.args(), max_new=2, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"), stream=0)
    usp.usp_check()
    check_attention(c, out, lse)
    o, z = usp.usp_paged_attn_q4(q, kc, vc, ks, vs, table[:0], cu[:1], kv[:0], out=torch.full_like(q.contiguous(), 3.0))
    usp.usp_check()
    assert (o == 3).all()
    usp.usp_paged_attn_q4(q[:0], kc, vc, ks, vs, table, cu * 0, kv)
    usp.usp_check()
