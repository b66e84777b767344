"""usp_paged_attn on data whose answer is known almost to the bit, so that a key that is lost, counted twice or taken
from another place shows however long the sequence is; lengths past the table; and both bf16 kernels in one call at
head dim 128."""
import random

import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from paged_ref import HALF_STEP, Cache, check_attention

pytestmark = pytest.mark.gpu


def class_of(kind, keys, hd):
    """The column in which key j's row of V is 1: its place modulo hd, in steps of 1, 16, 64, 100 or 1024 keys."""
    return torch.arange(keys) // kind % hd


def counted(c, kind):
    """K = 0 and V one-hot by place: every weight is 1, so o = (visible keys of the column) / (visible keys) and
    lse = log(visible keys). A key lost moves its column's count, and the lse by 1 / keys: 1.6e-5 at 60000."""
    c.k_cache.zero_()
    c.v_cache.fill_(float("nan"))
    for i, (kv, _) in enumerate(c.reqs):
        v = torch.nn.functional.one_hot(class_of(kind, kv, c.hd), c.hd).to(c.dtype).cuda()
        pages = -(-kv // c.ps)
        rows = torch.full((pages * c.ps, c.hd), float("nan"), dtype=c.dtype, device="cuda")
        rows[:kv] = v
        c.v_cache[c.table[i, :pages].long()] = rows.view(pages, 1, c.ps, c.hd).expand(-1, c.hkv, -1, -1)


def check_counted(c, out, lse, kind, causal=True):
    """The kernels' own roundings: the weights are 2^0 and the sums whole numbers below 2^24, exact in fp32 in any
    order; 1 / n and the product with it, or a division, 2^-23 in all; half a step of the output's type. lse: log2 to
    2 units in the last place (2^-22; the table of CUDA's math functions), times ln 2, two roundings more of 2^-24."""
    t = 0
    for kv, n in c.reqs:
        cls = torch.nn.functional.one_hot(class_of(kind, kv, c.hd), c.hd).cumsum(0)
        cls = torch.cat([torch.zeros(1, c.hd, dtype=torch.int64), cls]).cuda()
        see = (torch.arange(n, device="cuda") + kv - n + 1).clamp(0, kv) if causal else torch.full((n,), kv, device="cuda")
        want = torch.where(see[:, None] > 0, cls[see].double() / see[:, None].clamp(min=1), 0.0)[:, None]
        err = (out[t:t + n].double() - want).abs()
        assert (err <= want * (HALF_STEP[c.dtype] + 2.0 ** -22)).all(), (kv, n, (err / want.clamp(min=1e-9)).max().item())
        z = see.double().log()[:, None].expand(-1, c.hq)
        some = see > 0
        assert (lse[t:t + n][~some] == float("-inf")).all()
        zerr = (lse[t:t + n].double() - z)[some].abs()
        assert (zerr <= z[some] * (2.0 ** -22 + 2.0 ** -23)).all(), (kv, n, zerr.max().item())
        t += n


LONG = [[(60000, 1)], [(30, 1), (25000, 1), (27000, 2), (7, 0), (100, 1)], [(25000, 37), (300, 1)], [(131072, 1), (1, 1)]]
SHORT = [[(1, 1), (63, 1), (64, 1), (65, 1), (128, 1), (129, 1), (5000, 1)], [(300, 257), (2000, 64), (130, 130), (40, 60)],
         [(9000, 700)], [(700, 3), (4000, 5), (33, 33)]]
HEADS = [(8, 1, 128), (5, 1, 64), (6, 2, 64), (4, 4, 128), (20, 1, 128), (64, 1, 64), (32, 8, 128)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hkv,hd", HEADS)
@pytest.mark.parametrize("reqs", LONG + SHORT, ids=["60000", "some", "chunk", "131072", "tiles", "chunks", "one", "few"])
def test_every_key_counts_once(reqs, hq, hkv, hd, dt):
    c = Cache(reqs, hq, hkv, hd, 64, dt, seed=12)
    for kind in (1, 16, 64, 100, 1024):
        counted(c, kind)
        for causal in (True, False):
            out, lse = usp.usp_paged_attn(*c.args(), max_new=c.max_new, causal=causal)
            usp.usp_check()
            check_counted(c, out, lse, kind, causal)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [1, 3, 150])
def test_lengths_past_the_table_are_the_tables(dt, new):
    """kv_lens above what the table's columns hold counts as what they hold; a page outside the cache is zeros."""
    c = Cache([(600, new), (352, 2), (90, 1)], 4, 2, 64, 32, dt, seed=3, v_scale=0.5)
    width = c.table.shape[1]
    assert width * 32 > 600
    c.kv[0] = 2 ** 31 - 1
    c.kv[1] = width * 32 + 1
    for i in (0, 1):   # the columns behind the request's own hold no page: zero keys and values
        held = -(-c.reqs[i][0] // 32)
        last = torch.zeros(width * 32 - c.reqs[i][0], c.hkv, c.hd, dtype=dt)
        assert c.reqs[i][0] == held * 32 or i == 0
        if i == 0:     # the rest of its last page too
            page = int(c.table[0, held - 1])
            c.k_cache[page, :, 600 % 32:], c.v_cache[page, :, 600 % 32:] = 0, 0
        c.k[i], c.v[i] = torch.cat([c.k[i], last]), torch.cat([c.v[i], last])
        c.reqs[i] = (width * 32, c.reqs[i][1])
    for m in (None, 1):
        out = torch.full_like(c.q.contiguous(), float("nan"))
        out, lse = usp.usp_paged_attn(*c.args(), max_new=m, out=out)
        usp.usp_check()
        check_attention(c, out, lse)


@pytest.mark.parametrize("hq,hkv,chunks,singles", [(32, 8, 3, 90), (8, 8, 5, 70), (16, 16, 2, 40), (16, 2, 4, 300)])
def test_both_bf16_kernels_in_one_call_at_head_dim_128(hq, hkv, chunks, singles):
    """So many single tokens beside chunks that the kernel for few rows takes them in a launch of its own, second
    in the call: by the definition, to the same bits in a graph, and after work that is still writing the inputs."""
    r = random.Random(hq + singles)
    reqs = [(r.randrange(1, 3000), 1) for _ in range(singles)] + [(n + r.randrange(1500), n) for n in
                                                                  [r.randrange(100, 400) for _ in range(chunks)]]
    r.shuffle(reqs)
    c = Cache(reqs, hq, hkv, 128, 64, torch.bfloat16, seed=13)
    need = usp.usp_paged_attn_workspace_size(c.q, c.k_cache, c.table, c.max_new)
    few = usp.usp_paged_attn_workspace_size(c.q, c.k_cache, c.table, 1)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    args = [t.contiguous() for t in c.args()]
    out, lse = usp.usp_paged_attn(*args, max_new=c.max_new, workspace=ws)
    usp.usp_check()
    assert (ws[need - few:] != 0xff).any()   # the second kernel ran: it leaves its CTAs' headers
    check_attention(c, out, lse)
    live, slow = [torch.zeros_like(t) for t in args], torch.randn(2048, 2048, device="cuda")

    def work():
        for t in live:
            t.zero_()
        for _ in range(3):
            y = slow @ slow
        y.sum()
        for t, x in zip(live, args):
            t.copy_(x)
        return usp.usp_paged_attn(*live, max_new=c.max_new)
    got = work()
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = work()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)


def test_a_call_of_several_seconds():
    """One token over 400 million keys on every SM: no wait inside the kernel gives up while the keys before are
    still being worked on. (The table names one page over and over.)"""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    hkv, G, hd, ps, kv = sms, 33, 64, 256, 400_000_037
    k = torch.zeros(2, hkv, ps, hd, dtype=torch.bfloat16, device="cuda")
    v = torch.nn.functional.one_hot(torch.arange(ps) % hd, hd).to(k).expand(2, hkv, -1, -1).contiguous()
    table = torch.ones(1, -(-kv // ps), dtype=torch.int32, device="cuda")
    q = torch.randn(1, hkv * G, hd, device="cuda").to(torch.bfloat16)
    cu, kvs = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([kv], dtype=torch.int32, device="cuda")
    ws = torch.empty(usp.usp_paged_attn_workspace_size(q, k, table, 1), dtype=torch.uint8, device="cuda")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    out, lse = usp.usp_paged_attn(q, k, v, table, cu, kvs, max_new=1, workspace=ws)
    b.record()
    usp.usp_check()
    assert a.elapsed_time(b) > 2000     # as long as a wait may be that is not for a segment
    # exact sums: counts per column stay below 2^24, the normaliser is a multiple of 128 below 2^31 until its last tile;
    # then its rounding, 1 / l, the product (2^-24 each), log2 to 2 units in the last place and the product with ln 2
    want = torch.full((hd,), kv // hd, dtype=torch.float64, device="cuda")
    want[:kv % hd] += 1
    want /= kv
    err = (out[0].double() - want).abs()
    assert (err <= want * (HALF_STEP[torch.bfloat16] + 2.0 ** -21)).all()
    assert ((lse.double() - torch.log(torch.tensor(float(kv), dtype=torch.float64))).abs() <= 20 * 2.0 ** -21).all()
