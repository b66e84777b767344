"""usp_paged_attn_q4 on data whose answer is known almost to the bit, so that a key that is lost, counted twice or taken
from another place shows however long the sequence is; lengths past the table; both kernels in one call; very long calls."""
import random

import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from paged_ref import HALF_STEP, check_attention
from q4_ref import Q4Cache, pack
from test_gpu_paged_sharp import LONG, SHORT, check_counted, class_of

pytestmark = pytest.mark.gpu
ONE = 160  # the byte of a scale of 1: 8 * 2^(20 - 23)


def counted(c, kind):
    """K = 0 and V one-hot by place (see test_gpu_paged_sharp.counted); rows that no request owns keep their random bytes."""
    for i, (kv, _) in enumerate(c.reqs):
        page, row = c.table[i, torch.arange(kv, device="cuda") // c.ps].long(), torch.arange(kv, device="cuda") % c.ps
        v = pack(torch.nn.functional.one_hot(class_of(kind, kv, c.hd), c.hd).float()).cuda()
        c.k_cache[page, :, row] = 0
        c.v_cache[page, :, row] = v[:, None].expand(-1, c.hkv, -1)
        c.v_scales[page, :, row] = ONE


ROWS = [[(26000, 5), (400, 3), (129, 4)], [(5000, 8), (0, 2), (64, 8)], [(26000, 16), (127, 9), (1, 1), (700, 12)]]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hkv,hd", [(8, 1, 128), (5, 1, 64), (6, 2, 64), (4, 4, 128), (20, 1, 128), (40, 1, 64), (16, 4, 128)])
@pytest.mark.parametrize("reqs", LONG + SHORT + ROWS, ids=["60000", "some", "chunk", "131072", "tiles", "chunks", "one", "few",
                                                           "five", "eight", "sixteen"])
def test_every_key_counts_once(reqs, hq, hkv, hd, dt):
    c = Q4Cache(reqs, hq, hkv, hd, 64, dt, seed=12)
    for kind in (1, 16, 64, 100, 1024):
        counted(c, kind)
        for causal in (True, False):
            out, lse = usp.usp_paged_attn_q4(*c.args(), max_new=c.max_new, causal=causal)
            usp.usp_check()
            check_counted(c, out, lse, kind, causal)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [1, 3, 9, 150])
def test_lengths_past_the_table_are_the_tables(dt, new):
    """kv_lens above what the table's columns hold counts as what they hold; a page outside the cache is zeros."""
    c = Q4Cache([(600, new), (352, 2), (90, 1)], 4, 2, 64, 32, dt, seed=3)
    width = c.table.shape[1]
    assert width * 32 > 600
    c.kv[0] = 2 ** 31 - 1
    c.kv[1] = width * 32 + 1
    for i in (0, 1):   # the columns behind the request's own hold no page: zero keys and values
        last = torch.zeros(width * 32 - c.reqs[i][0], c.hkv, c.hd).double()
        if i == 0:     # the rest of its last page too
            page = int(c.table[0, -(-600 // 32) - 1])
            c.k_cache[page, :, 600 % 32:], c.v_cache[page, :, 600 % 32:] = 0, 0
        c.k[i], c.v[i] = torch.cat([c.k[i], last]), torch.cat([c.v[i], last])
        c.reqs[i] = (width * 32, c.reqs[i][1])
    for m in (None, 1):
        out = torch.full_like(c.q.contiguous(), float("nan"))
        out, lse = usp.usp_paged_attn_q4(*c.args(), max_new=m, out=out)
        usp.usp_check()
        check_attention(c, out, lse)


@pytest.mark.parametrize("hq,hkv,hd,chunks,singles", [(32, 8, 128, 3, 90), (8, 8, 64, 5, 70), (48, 3, 128, 2, 40), (16, 2, 64, 4, 300)])
def test_both_kernels_in_one_call(hq, hkv, hd, chunks, singles):
    """Single tokens beside chunks: by the definition, to the same bits in a graph, and after work that is still writing the
    inputs."""
    r = random.Random(hq + singles)
    reqs = [(r.randrange(1, 3000), 1) for _ in range(singles)] + [(n + r.randrange(1500), n) for n in
                                                                  [r.randrange(100, 400) for _ in range(chunks)]]
    r.shuffle(reqs)
    c = Q4Cache(reqs, hq, hkv, hd, 64, torch.bfloat16, seed=13)
    args = [t.contiguous() for t in c.args()]
    out, lse = usp.usp_paged_attn_q4(*args, max_new=c.max_new)
    usp.usp_check()
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
        return usp.usp_paged_attn_q4(*live, max_new=c.max_new)
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


@pytest.mark.parametrize("G,kv", [(1, 1_050_000_037), (12, 700_000_037), (33, 400_000_037)])
def test_a_call_of_several_seconds(G, kv):
    """One token over hundreds of millions of keys for every SM: no wait inside the kernels gives up while the keys before
    are still being worked on. (The table names one page over and over.)"""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    hkv, hd, ps = sms, 64, 256
    k = torch.zeros(2, hkv, ps, hd // 2, dtype=torch.uint8, device="cuda")
    v = pack(torch.nn.functional.one_hot(torch.arange(ps) % hd, hd).float()).cuda().expand(2, hkv, -1, -1).contiguous()
    s = torch.full((2, hkv, ps, hd // 32), ONE, dtype=torch.uint8, device="cuda")
    table = torch.ones(1, -(-kv // ps), dtype=torch.int32, device="cuda")
    q = torch.randn(1, hkv * G, hd, device="cuda").to(torch.bfloat16)
    cu, kvs = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([kv], dtype=torch.int32, device="cuda")
    out, lse = usp.usp_paged_attn_q4(q, k, v, s, s, table, cu, kvs, max_new=1)   # 2 to 3 seconds
    usp.usp_check()
    # exact sums: counts per column stay below 2^24, normalisers whole numbers that the fp32 sums of lanes, warps and CTAs hold
    # to 2^-24 each (a dozen of them); 1 / l, the product (2^-24 each), log2 to 2 units in the last place and the product with ln 2
    want = torch.full((hd,), kv // hd, dtype=torch.float64, device="cuda")
    want[:kv % hd] += 1
    want /= kv
    err = (out[0].double() - want).abs()
    assert (err <= want * (HALF_STEP[torch.bfloat16] + 2.0 ** -20)).all()
    assert ((lse.double() - torch.log(torch.tensor(float(kv), dtype=torch.float64))).abs() <= 20 * 2.0 ** -20).all()
