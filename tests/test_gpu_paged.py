"""The paged K/V cache: page plan, cache append and the attention over the cache, against plain 64-bit
definitions with bounds derived from the roundings the kernels make (tests/paged_ref.py)."""
import math
import random

import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from paged_ref import Cache, check_attention, plan_ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- plan ----------------------------------------------------------------------------------------
def run_plan(ctx, new, free, head, table, ps, num_pages, max_tokens):
    t = i32(table).view(len(ctx), -1)
    outs = usp.usp_page_plan(i32(ctx), i32(new), i32(free), i32([head]), t, ps, num_pages, max_tokens)
    usp.usp_check()
    got = [t.tolist()] + [x.tolist() for x in outs]
    want = plan_ref(ctx, new, free, head, table, ps, num_pages, max_tokens)
    for name, g, w in zip(("table", "slots", "cu", "kv", "counts"), got, want):
        assert list(g) == list(w), name


def random_plan(nreq, ctx_hi, new_hi, ps, seed, spare=0, width_less=0, tokens_more=0):
    r = random.Random(seed)
    ctx = [r.choice([0, r.randint(0, ctx_hi), ps * r.randint(0, ctx_hi // ps)]) for _ in range(nreq)]
    new = [r.choice([0, 1, r.randint(0, new_hi)]) for _ in range(nreq)]
    old = [-(-c // ps) for c in ctx]
    every = [-(-(c + n) // ps) for c, n in zip(ctx, new)]
    num = sum(every) + 7
    ids = list(range(num))
    r.shuffle(ids)
    width = max(max(every) - width_less, 1)
    table, at = [], 0
    for o in old:
        row = ids[at:at + o][:width]
        at += o
        table.append(row + [-7] * (width - len(row)))
    fresh = sum(every) - sum(old)
    free = [99999] * 2 + ids[at:at + max(0, fresh + spare)]
    return ctx, new, free, 2, table, ps, num, max(0, sum(new) + tokens_more)


@pytest.mark.parametrize("nreq,ctx_hi,new_hi,ps", [(1, 40, 3, 16), (3, 0, 70, 16), (64, 900, 1, 64), (64, 900, 200, 32),
                                                   (256, 3000, 64, 128), (1500, 50, 9, 16), (2049, 600, 3, 256)])
def test_plan_matches_definition(nreq, ctx_hi, new_hi, ps):
    run_plan(*random_plan(nreq, ctx_hi, new_hi, ps, seed=nreq, spare=3))


@pytest.mark.parametrize("spare,width_less,tokens_more", [(-3, 0, 0), (0, 2, 0), (0, 0, 300), (0, 0, -5), (-100000, 1, 11)])
def test_plan_shortages(spare, width_less, tokens_more):
    """Pages, columns or slots that run out: -1 slots, counted; everything else as it would be."""
    run_plan(*random_plan(70, 500, 40, 16, seed=9, spare=spare, width_less=width_less, tokens_more=tokens_more))


def test_plan_odd_values():
    run_plan([5, -3, 0, 20], [-1, 4, 0, 13], [3, 1, 2, 9, -4, 77], 0, [[50, 51, 52, 53]] * 4, 16, 60, 40)
    run_plan([0], [1000], list(range(100)), 0, [[-1] * 70], 16, 10, 1000)  # page ids at and above num_pages
    run_plan([0, 0], [0, 0], [], 0, [[-1], [-1]], 16, 4, 0)


def test_plan_runs_again_and_goes_on():
    """The same inputs give the same outputs, and the outputs are the next step's inputs."""
    r = random.Random(3)
    ps, nreq, width = 16, 20, 30
    free = list(range(400))
    r.shuffle(free)
    ctx, table, head = [0] * nreq, [[-1] * width for _ in range(nreq)], 0
    d_ctx, d_table, d_head, d_free = i32(ctx), i32(table), i32([0]), i32(free)
    for step in range(4):
        new = [r.choice([0, 1, r.randint(0, 60)]) for _ in range(nreq)]
        a = usp.usp_page_plan(d_ctx, i32(new), d_free, d_head, d_table, ps, 400, sum(new) + 3)
        b = usp.usp_page_plan(d_ctx, i32(new), d_free, d_head, d_table, ps, 400, sum(new) + 3)
        usp.usp_check()
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        table, slots, cu, kv, counts = plan_ref(ctx, new, free, head, table, ps, 400, sum(new) + 3)
        assert d_table.tolist() == table and a[0].tolist() == slots and a[3].tolist() == counts
        d_ctx, d_head, ctx, head = a[2], a[3][1:2], kv, counts[1]


# ---- append ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,hkv,hd,ps,dt", [(1, 1, 64, 16, torch.bfloat16), (77, 8, 128, 64, torch.bfloat16),
                                                 (1001, 3, 64, 32, torch.float32), (5000, 2, 128, 256, torch.float32),
                                                 (40000, 8, 128, 16, torch.bfloat16)])
@pytest.mark.parametrize("strided", [False, True])
def test_append_is_a_bit_exact_scatter(tokens, hkv, hd, ps, dt, strided):
    g = torch.Generator().manual_seed(tokens)
    pages = -(-tokens // ps) + 4
    slots = torch.randperm(pages * ps, generator=g)[:tokens].to(torch.int32)
    slots[torch.rand(tokens, generator=g) < 0.1] = -1
    if tokens > 3:
        slots[1], slots[2] = pages * ps, 2 ** 31 - 1      # one past the cache, and far past it
    row = hkv * hd
    both = torch.randn(tokens, 2 * row + (16 if strided else 0), generator=g).to(dt).cuda()
    k, v = both[:, :row].unflatten(1, (hkv, hd)), both[:, row:2 * row].unflatten(1, (hkv, hd))
    buf = torch.randn(pages, 2, hkv, ps, hd, generator=g).to(dt).cuda()
    kc, vc = buf[:, 0], buf[:, 1]
    if not strided:
        k, v, kc, vc = k.contiguous(), v.contiguous(), kc.contiguous(), vc.contiguous()
    want_k, want_v = kc.clone(), vc.clone()
    ok = (slots >= 0) & (slots < pages * ps)
    page, at = (slots[ok] // ps).long().cuda(), (slots[ok] % ps).long().cuda()
    want_k[page, :, at], want_v[page, :, at] = k[ok.cuda()], v[ok.cuda()]
    usp.usp_cache_append(k, v, kc, vc, slots.cuda())
    usp.usp_check()
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


# ---- attention ------------------------------------------------------------------------------------
DECODE = [(1, 1), (17, 1), (64, 1), (65, 1), (0, 0), (300, 1), (0, 1), (1000, 1), (5, 0), (128, 1)]
CHUNKS = [(1, 1), (130, 130), (129, 2), (300, 257), (0, 0), (700, 64), (65, 65), (1000, 1), (400, 33)]
# fewer keys than new tokens: the first rows see nothing
SHORT = [(3, 40), (0, 7), (200, 300), (1, 2)]


def attend(c, **kw):
    # poisoned outputs: every row of a request has to be written
    kw.setdefault("out", torch.full_like(c.q.contiguous(), float("nan")))
    kw.setdefault("lse", torch.full(c.q.shape[:2], float("nan"), device="cuda"))
    r = usp.usp_paged_attn(*c.args(), **kw)
    usp.usp_check()
    return r


@pytest.mark.parametrize("reqs", [DECODE, CHUNKS, SHORT, [(4000, 1)], [(3001, 500)], [(257, 257)]],
                         ids=["decode", "chunks", "short", "one-decode", "one-chunk", "one-prompt"])
@pytest.mark.parametrize("hq,hkv,hd,ps,dt", [
    (8, 2, 128, 16, torch.bfloat16), (4, 4, 64, 64, torch.bfloat16), (8, 1, 128, 128, torch.bfloat16),
    (10, 2, 64, 32, torch.bfloat16), (7, 1, 128, 256, torch.bfloat16), (32, 1, 64, 16, torch.bfloat16),
    (128, 1, 128, 64, torch.bfloat16), (4, 2, 64, 16, torch.float32), (3, 1, 128, 256, torch.float32),
    (16, 1, 64, 32, torch.float32)])
def test_attention_matches_definition(reqs, hq, hkv, hd, ps, dt):
    c = Cache(reqs, hq, hkv, hd, ps, dt, seed=hq + hd)
    out, lse = attend(c, max_new=c.max_new)
    check_attention(c, out, lse)
    # without the host's bound, and with one that is too small: the same definition
    for m in (None, 1):
        out, lse = attend(c, max_new=m)
        check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("reqs", [DECODE, CHUNKS, SHORT], ids=["decode", "chunks", "short"])
def test_attention_without_the_causal_mask(reqs, dt):
    c = Cache(reqs, 8, 2, 64, 32, dt, seed=1)
    out, lse = attend(c, causal=False, scale=0.3)
    check_attention(c, out, lse, causal=False, scale=0.3)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("reqs", [DECODE, CHUNKS], ids=["decode", "chunks"])
def test_attention_strides_and_foreign_rows(reqs, dt):
    """q and out as slices of wider rows, an interleaved cache, a wider table; rows of no request and the
    columns beside out keep their bytes."""
    c = Cache(reqs, 8, 2, 128, 16, dt, seed=2, interleave=True, qpad=64)
    T, hq, hd = c.q.shape
    wide = torch.full((T + 9, hq * hd + 32), 7.0, dtype=dt, device="cuda")
    q = torch.full((T + 9, hq * hd + 64), float("nan"), dtype=dt, device="cuda")
    q[4:4 + T, :hq * hd] = c.q.flatten(1)
    lse = torch.full((T + 9, hq), 7.0, device="cuda")
    table = torch.full((c.table.shape[0], c.table.shape[1] + 5), 2 ** 30, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    out = wide[:, :hq * hd].unflatten(1, (hq, hd))
    usp.usp_paged_attn(q[:, :hq * hd].unflatten(1, (hq, hd)), c.k_cache, c.v_cache, table[:, :c.table.shape[1]],
                       c.cu + 4, c.kv, out=out, lse=lse)
    usp.usp_check()
    check_attention(c, out[4:4 + T], lse[4:4 + T])
    assert (wide[:4] == 7).all() and (wide[4 + T:] == 7).all() and (wide[:, hq * hd:] == 7).all()
    assert (lse[:4] == 7).all() and (lse[4 + T:] == 7).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [1, 150])
def test_attention_pages_outside_the_cache_read_as_zeros(dt, new):
    """Wrong page ids and lengths past the table: no fault; such pages hold zero keys and values."""
    c = Cache([(600, new), (90, 1)], 4, 2, 64, 32, dt, seed=3)
    bad = {1: -1, 4: c.k_cache.shape[0], 6: 2 ** 31 - 1, 7: -2 ** 31}
    for col, page in bad.items():
        c.table[0, col] = page
        c.k[0][col * 32:(col + 1) * 32] = 0
        c.v[0][col * 32:(col + 1) * 32] = 0
    out, lse = attend(c)
    check_attention(c, out, lse)
    width = c.table.shape[1]
    c.kv[1] = 2 ** 31 - 1                      # more keys than the table has room for
    c.table[1] = c.table[0]
    c.table[1, -1] = 0
    out, lse = attend(c)
    assert out.shape == c.q.shape and width * 32 >= 600


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_attention_many_requests(dt):
    r = random.Random(4)
    reqs = [(k, min(k, r.choice([0, 1, 1, 1, 2, 30]))) for k in (r.choice([0, 1, 16, 33, 90]) for _ in range(2500))]
    c = Cache(reqs, 4, 2, 64, 16, dt, seed=4)
    out, lse = attend(c)
    check_attention(c, out, lse)


def test_attention_peaked_and_large_scores():
    """Scores up to some hundred: one key takes all the weight, and the running maximum keeps moving."""
    for dt in (torch.bfloat16, torch.float32):
        c = Cache([(900, 1), (500, 200), (64, 64)], 8, 2, 128, 64, dt, seed=5)
        c.q.mul_(24)
        out, lse = attend(c)
        check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hkv,hd", [(8, 1, 128), (5, 1, 64), (6, 2, 64)])
@pytest.mark.parametrize("reqs", [[(60000, 1)], [(30, 1), (25000, 1), (27000, 2), (7, 0), (100, 1)], [(25000, 37), (300, 1)]],
                         ids=["one", "some", "chunk"])
def test_attention_units_of_many_parts(reqs, hq, hkv, hd, dt):
    """Long sequences with few KV heads: a row's keys lie over most of the GPU, in up to 304 parts."""
    c = Cache(reqs, hq, hkv, hd, 64, dt, seed=10)
    out, lse = attend(c, max_new=c.max_new)
    check_attention(c, out, lse)


@pytest.mark.parametrize("hq,hkv,hd", [(8, 8, 64), (16, 4, 128), (24, 3, 64), (64, 2, 128), (128, 1, 128), (12, 4, 128)])
def test_attention_long_prompts(hq, hkv, hd):
    """Enough blocks that out is written in boxes where a warp's rows are whole: every grouping, blocks that end
    inside a warp's rows, and rows of other requests and columns beside out that stay as they were."""
    T = 160 * 2 * 256 * hkv // hq // hkv + 700      # more than two units of 256 rows for each of up to 160 SMs
    c = Cache([(T, T), (333, 129), (65, 65)], hq, hkv, hd, 128, torch.bfloat16, seed=11)
    wide = torch.full((c.T + 5, hq * hd + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :hq * hd].unflatten(1, (hq, hd))
    lse = torch.full((c.T + 5, hq), 7.0, device="cuda")
    q = torch.cat([c.q.contiguous(), c.q[:5]])
    usp.usp_paged_attn(q, c.k_cache, c.v_cache, c.table, c.cu, c.kv, out=out, lse=lse)
    usp.usp_check()
    assert (wide[:, hq * hd:] == 7).all() and (wide[c.T:] == 7).all() and (lse[c.T:] == 7).all()
    assert not (out[:c.T] == 7).all(-1).any() and (lse[:c.T] != 7).all()
    # the long request in the definition's memory: its last rows only, as a chunk of their own
    n = 300
    tail = Cache.__new__(Cache)
    tail.__dict__.update(c.__dict__)
    tail.reqs, tail.q, tail.T = [(T, n), (333, 129), (65, 65)], c.q[T - n:], c.T - T + n
    check_attention(tail, out[T - n:c.T], lse[T - n:c.T])
    head = Cache.__new__(Cache)
    head.__dict__.update(c.__dict__)
    head.reqs, head.q, head.T, head.k, head.v = [(n, n)], c.q[:n], n, [c.k[0][:n]], [c.v[0][:n]]
    check_attention(head, out[:n], lse[:n])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("reqs", [[(200, 2000)], [(300, 40)] + [(0, 40)] * 30 + [(300, 40)], [(0, 90)] * 9,
                                  [(1, 500), (900, 40), (2, 700), (0, 50), (40, 1)]],
                         ids=["one-request", "between", "only", "mixed"])
def test_attention_runs_of_units_without_a_key(reqs, dt):
    """Many blocks of tokens in a row that see no key (more new tokens than keys), before, between and behind
    blocks that do."""
    c = Cache(reqs, 8, 2, 64, 32, dt, seed=9)
    for kw in (dict(max_new=c.max_new), dict(max_new=1), dict(max_new=c.max_new, causal=False)):
        out, lse = attend(c, **kw)
        check_attention(c, out, lse, causal=kw.get("causal", True))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("reqs", [[(500, 1), (64, 1), (9000, 1)], [(300, 150), (2000, 70), (80, 80)]], ids=["decode", "chunks"])
def test_attention_a_nan_query_row_is_nan_and_stays_alone(reqs, dt):
    """A query row that holds a NaN gets NaN in out and lse, in units that one CTA finishes and in cut ones;
    every other row stays what it is. (Not to the bit: rows of a unit rescale together when the maximum of one
    of them grows, so a row's rounding depends on its neighbours' scores; the bounds count any such order.)"""
    c = Cache(reqs, 8, 2, 64, 32, dt, seed=8)
    q = c.q.clone()
    want = [x.clone() for x in attend(c)]
    rows = [(0, 3), (c.T // 2, 6), (c.T - 1, 0)]
    for t, h in rows:
        c.q[t, h, 5] = float("nan")
    out, lse = attend(c)
    hit = torch.zeros(c.T, c.hq, dtype=torch.bool, device="cuda")
    for t, h in rows:
        hit[t, h] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    out[hit], lse[hit], c.q = want[0][hit], want[1][hit], q
    check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_attention_same_bits_on_every_run(dt):
    c = Cache([(5000, 1), (3000, 300), (40, 40), (2500, 1)], 8, 2, 128, 16, dt, seed=6)
    a = [x.clone() for x in attend(c)]
    for _ in range(3):
        b = attend(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_on_another_stream_and_in_a_graph():
    """On a side stream with the call's own allocations; captured, and replayed with other lengths."""
    c = Cache([(700, 1), (90, 1), (1300, 1)], 8, 2, 128, 16, torch.bfloat16, seed=7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = usp.usp_paged_attn(*c.args(), max_new=1, stream=s)
    s.synchronize()
    check_attention(c, out, lse)
    out2, lse2 = usp.usp_paged_attn(*c.args(), max_new=1, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go, gl = usp.usp_paged_attn(*c.args(), max_new=1)
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


# ---- together -------------------------------------------------------------------------------------
@pytest.mark.parametrize("hq,hkv,hd,ps,dt", [(8, 2, 128, 64, torch.bfloat16), (4, 4, 64, 16, torch.float32)])
def test_prompt_chunks_and_tokens_through_the_cache(hq, hkv, hd, ps, dt):
    """A serving loop: prompts in chunks, then token by token; plan, append, attention each step. Every
    step agrees with the definition, and the whole of it with usp_forward over the finished sequences."""
    from paged_ref import HALF_STEP, attention64
    g = torch.Generator().manual_seed(8)
    L = [520, 300]
    nreq, num = 2, 64
    r = [[torch.randn(n, h, hd, generator=g).to(dt).cuda() for h in (hq, hkv, hkv)] for n in L]
    kc = torch.full((num, hkv, ps, hd), float("nan"), dtype=dt, device="cuda")
    vc = kc.clone()
    table = torch.full((nreq, 40), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(num, generator=g).to(torch.int32).cuda()
    head, ctx = i32([0]), i32([0, 0])
    outs, lses, at = [[], []], [[], []], [0, 0]
    steps = [[257, 100], [200, 0], [60, 199]] + [[1, 1]] + [[1, 0]] * 2
    for new in steps:
        T = sum(new)
        q, k, v = [torch.cat([r[i][x][at[i]:at[i] + new[i]] for i in range(nreq)]) for x in range(3)]
        slots, cu, kv, counts = usp.usp_page_plan(ctx, i32(new), free, head, table, ps, num, T + 5)
        usp.usp_cache_append(k, v, kc, vc, slots[:T])
        o, z = usp.usp_paged_attn(q, kc, vc, table, cu, kv, max(new))
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
        reqs, q, T = [(n, n) for n in L], torch.cat([x[0] for x in r]), sum(L)
        k, v = [x[1] for x in r], [x[2] for x in r]
    Whole.hq, Whole.hkv, Whole.hd, Whole.dtype = hq, hkv, hd, dt
    out, lse = torch.cat(outs[0] + outs[1]), torch.cat(lses[0] + lses[1])
    check_attention(Whole, out, lse)
    _, _, bo, bl = attention64(Whole)
    t = 0
    for i, n in enumerate(L):
        fo, fl = usp.usp_attention(*[x[None] for x in r[i]], ud=1, rd=1)
        usp.usp_check()
        # two computations, each within its bound of the definition
        assert ((fo[0].double() - out[t:t + n].double()).abs() <= 2 * bo[t:t + n] + HALF_STEP[dt]).all()
        assert ((fl[0].double() - lse[t:t + n].double()).abs() <= 2 * bl[t:t + n] + 1e-5).all()
        t += n


def test_parts_of_a_sequence_merge():
    """Two caches with half of the keys each: the partials merge (usp_lse_merge) to the whole."""
    c = Cache([(1000, 1), (640, 1)], 8, 2, 128, 64, torch.float32, seed=9)
    parts = []
    for lo, hi in ((0, 320), (320, None)):
        kv = i32([len(c.k[i][lo:hi]) for i in range(2)])
        table = c.table[:, lo // 64:].contiguous() if lo else c.table
        o, z = usp.usp_paged_attn(c.q, c.k_cache, c.v_cache, table, c.cu, kv, 1, causal=False)
        parts.append((o, z))
    usp.usp_lse_merge(parts[0][0], parts[0][1], parts[1][0], parts[1][1])
    usp.usp_check()
    # the merge adds a few roundings of its own (weights and products in fp32)
    class Both:
        pass
    o, z = parts[0]
    from paged_ref import attention64
    ref, lref, bo, bl = attention64(c, causal=False)
    assert ((o.double() - ref).abs() <= 3 * bo + 2.0 ** -20 * ref.abs()).all()
    assert ((z.double() - lref).abs() <= 3 * bl + 2.0 ** -20).all()
    assert math.isfinite(z.sum().item())


# ---- at the edges of what the calls allow ----------------------------------------------------------
def test_attention_fewer_tokens_than_a_tile_of_queries():
    """One short chunk alone: the query tile's box is taller than q."""
    for new, hq, hkv, hd in ((9, 8, 2, 128), (17, 2, 2, 64), (33, 1, 1, 128), (3, 64, 2, 64)):
        c = Cache([(new + 60, new)], hq, hkv, hd, 16, torch.bfloat16, seed=new)
        out, lse = attend(c, max_new=new)
        check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_attention_shared_pages(dt):
    """Requests that begin with the same pages (a shared prompt) and go on in their own."""
    c = Cache([(300, 1), (290, 40), (256, 1)], 8, 2, 64, 64, dt, seed=21)
    for i in (1, 2):
        c.table[i, :4] = c.table[0, :4]
        c.k[i][:256], c.v[i][:256] = c.k[0][:256], c.v[0][:256]
    out, lse = attend(c)
    check_attention(c, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [1, 70])
def test_offsets_past_32_bits(dt, new):
    """A cache of more than 2^31 elements (and 2^32 bytes): append to and attend over its last pages."""
    hkv, ps, hd, num = 8, 256, 128, 8300
    kc, vc = (torch.empty(num, hkv, ps, hd, dtype=dt, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    c = Cache([(600, new), (256, new)], 16, hkv, hd, ps, dt, seed=22)
    pages = [[num - 1, num - 5, num - 3], [num - 2]]
    c.table = i32([pages[0], pages[1] + [-1, -1]])
    keys = torch.cat(c.k).cuda(), torch.cat(c.v).cuda()
    slots = i32([pages[i][p // ps] * ps + p % ps for i, (n, _) in enumerate(c.reqs) for p in range(n)])
    usp.usp_cache_append(*keys, kc, vc, slots)
    c.k_cache, c.v_cache = kc, vc
    out, lse = attend(c)
    check_attention(c, out, lse)


def test_two_calls_at_once_with_their_own_workspaces():
    cs = [Cache([(3000 + 100 * i, 1), (700, 90)], 8, 2, 128, 16, torch.bfloat16, seed=30 + i) for i in range(2)]
    alone = [[x.clone() for x in attend(c)] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [usp.usp_paged_attn(*c.args(), stream=s) for c, s in zip(cs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_calls_on_three_streams_keep_their_bits():
    """Calls of every kind running beside each other, so that kernels of several calls share an SM: each
    gives the bits that it gives alone."""
    r = random.Random(1)

    def make(i):
        reqs = [[(r.randrange(1, 4000), 1) for _ in range(r.randrange(1, 40))],
                [(r.randrange(300, 3000), r.randrange(1, 300)) for _ in range(r.randrange(1, 5))],
                [(r.randrange(100, 2500),) * 2 for _ in range(r.randrange(1, 4))],
                [(r.randrange(200, 3000), r.choice([1, 1, 1, 200])) for _ in range(20)]][i % 4]
        hkv = r.choice([1, 2, 4])
        c = Cache(reqs, hkv * r.choice([1, 2, 4, 5, 8]), hkv, r.choice([64, 128]), r.choice([16, 64, 256]),
                  torch.float32 if i % 5 == 4 else torch.bfloat16, seed=i)
        return c, [x.clone() for x in attend(c, max_new=c.max_new)]
    calls, streams = [make(i) for i in range(24)], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(600):
        wrong = []
        for _ in range(40):
            c, want = r.choice(calls)
            with torch.cuda.stream(r.choice(streams)):
                out, lse = torch.full_like(want[0], float("nan")), torch.full_like(want[1], float("nan"))
                usp.usp_paged_attn(*c.args(), max_new=c.max_new, out=out, lse=lse)
                wrong.append((out != want[0]).sum() + (lse != want[1]).sum())
        torch.cuda.synchronize()
        assert sum(int(x) for x in wrong) == 0
    usp.usp_check()


def test_whole_step_in_one_graph():
    """Plan, append and attention captured together and replayed for other lengths, with -1 slots behind
    the last token."""
    hq, hkv, hd, ps, num, cap = 8, 2, 64, 16, 80, 64
    g = torch.Generator().manual_seed(40)
    c = Cache([(0, 0), (0, 0)], hq, hkv, hd, ps, torch.bfloat16)
    kc, vc = (torch.full((num, hkv, ps, hd), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, free = torch.full((2, 30), -1, dtype=torch.int32, device="cuda"), torch.arange(num, dtype=torch.int32, device="cuda")
    ctx, new, head = i32([0, 0]), i32([0, 0]), i32([0])
    q, k, v = (torch.zeros(cap, h, hd, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))

    def step():
        slots, cu, kv, counts = usp.usp_page_plan(ctx, new, free, head, table, ps, num, cap)
        usp.usp_cache_append(k, v, kc, vc, slots)
        return (*usp.usp_paged_attn(q, kc, vc, table, cu, kv), kv, counts)
    step()
    usp.usp_check()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, kv, counts = step()
    c.k, c.v, c.q = [torch.empty(0, hkv, hd, dtype=torch.bfloat16)] * 2, [torch.empty(0, hkv, hd, dtype=torch.bfloat16)] * 2, q
    for lens in ([40, 13], [1, 1], [0, 50], [30, 0]):
        T = sum(lens)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).to(t.dtype))
        new.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for i, n in enumerate(lens):
            c.k[i], c.v[i] = torch.cat([c.k[i], k[at:at + n].cpu()]), torch.cat([c.v[i], v[at:at + n].cpu()])
            at += n
        c.reqs, c.T = [(len(c.k[i]), lens[i]) for i in range(2)], T
        c.q = q[:T]
        check_attention(c, out[:T], lse[:T])
        assert counts.tolist()[0] == T and counts.tolist()[2] == 0
        ctx.copy_(kv)
        head.copy_(counts[1:2])


def test_no_work_after_a_recorded_timeout_until_it_is_checked():
    from sequence_long_context_zigzag_gb300 import _abi
    c = Cache([(500, 1), (300, 80)], 8, 2, 128, 16, torch.bfloat16, seed=50)
    _abi.check("usp_selftest_timeout", _abi.load().usp_selftest_timeout(1000, torch.cuda.current_stream().cuda_stream))
    with pytest.raises(usp.UspError) as e:
        attend(c)
    assert e.value.status == _abi.USP_ERR_TIMEOUT
    out, lse = attend(c)
    check_attention(c, out, lse)


def test_binding_refuses_on_the_gpu():
    c = Cache([(50, 2), (20, 1)], 4, 2, 64, 16, torch.bfloat16)
    q, kc, vc, table, cu, kv = c.args()
    for bad in (dict(lse=torch.empty(3, 5, device="cuda")), dict(out=torch.empty(3, 4, 128, device="cuda")),
                dict(workspace=torch.empty(10, dtype=torch.uint8)), dict(lse=torch.empty(c.T, 4))):
        with pytest.raises(ValueError):
            usp.usp_paged_attn(*c.args(), **bad)
    with pytest.raises(ValueError, match="one device"):
        usp.usp_paged_attn(q, kc, vc, table.cpu(), cu, kv)
    with pytest.raises(usp.UspError):
        usp.usp_paged_attn(*c.args(), max_new=-1)
    with pytest.raises(usp.UspError):
        usp.usp_paged_attn(*c.args(), workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(usp.UspError):   # pages of 8 tokens
        usp.usp_paged_attn(q, kc[:, :, :8].contiguous(), vc[:, :, :8].contiguous(), table, cu, kv)
    with pytest.raises(ValueError):
        usp.usp_cache_append(q[:, :2], q[:, :2], kc, vc, i32([0]))
    n = usp.usp_paged_attn_workspace_size(q, kc, table, 2)
    out, lse = usp.usp_paged_attn(*c.args(), max_new=2, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"), stream=0)
    usp.usp_check()
    check_attention(c, out, lse)
    # no request, no token
    o, z = usp.usp_paged_attn(q, kc, vc, table[:0], cu[:1], kv[:0], out=torch.full_like(q.contiguous(), 3.0))
    usp.usp_check()
    assert (o == 3).all()
    usp.usp_paged_attn(q[:0], kc, vc, table, cu * 0, kv)
    usp.usp_check()


def test_calls_follow_the_work_before_them():
    """The kernels may start before the work before them in the stream has ended: inputs that long kernels,
    copies and other streams are still writing when the calls are made have to be seen, eagerly and in a
    graph."""
    hq, hkv, hd, ps = 8, 2, 128, 16
    for reqs in ([(700, 1), (90, 1)], [(600, 120), (90, 1)]):
        for dt in (torch.bfloat16, torch.float32):
            c = Cache(reqs, hq, hkv, hd, ps, dt, seed=60)
            want = [x.clone() for x in attend(c)]
            true = [t.clone() for t in c.args()]
            slow = torch.randn(4096, 4096, device="cuda")
            buf = [torch.empty_like(t) for t in true]
            rows = torch.arange(c.T, device="cuda", dtype=torch.int32)
            side = torch.cuda.Stream()
            dst = [torch.zeros(64, hkv, ps, hd, dtype=dt, device="cuda") for _ in range(2)]
            kvrows = [torch.randn(c.T, hkv, hd, device="cuda").to(dt) for _ in range(2)]
            late = [torch.zeros_like(x) for x in kvrows]

            def work():
                for d in dst:
                    d.zero_()
                for b, x in zip(late, kvrows):
                    b.zero_()
                for b, t in zip(buf, true):
                    b.zero_() if b.dtype == torch.int32 else b.fill_(1)
                here = torch.cuda.current_stream()
                side.wait_stream(here)
                with torch.cuda.stream(side):
                    (slow @ slow).sum()
                    buf[2].copy_(true[2])
                for _ in range(3):
                    y = slow @ slow
                y.sum()
                for i in (0, 1, 3, 4, 5):
                    buf[i].copy_(true[i])
                here.wait_stream(side)
                o1 = usp.usp_paged_attn(*buf)                       # after a copy and another stream
                for b, x in zip(late, kvrows):
                    b.copy_(x)
                usp.usp_cache_append(*late, *dst, rows)             # after a copy kernel
                p1 = usp.usp_page_plan(buf[5], buf[5], rows, rows[:1], buf[3].clone(), ps, 2 ** 20, 5000)
                o2 = usp.usp_paged_attn(*buf)                       # after its own kind
                return o1, p1, o2

            def check(o1, p1, o2):
                for o in (o1, o2):
                    assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
                assert torch.equal(p1[2], true[5] * 2)
                for d, x in zip(dst, kvrows):
                    assert torch.equal(d.transpose(1, 2).reshape(-1, hkv, hd)[:c.T], x)
            for _ in range(3):
                r = work()
                torch.cuda.synchronize()
                check(*r)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                r = work()
            for _ in range(3):
                g.replay()
                torch.cuda.synchronize()
                check(*r)
