"""Refusals of the rotation's and the 4-bit cache's calls, at the C ABI and in the binding, without a GPU: every case is
rejected before a launch."""
import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp
from sequence_long_context_zigzag_gb300 import _abi

GOOD, BAD = 0x10000, 0x10001   # never dereferenced
E = _abi


def make(cls, base, kw):
    base.update(kw)
    return cls(*[base[f] for f, _ in cls._fields_])


def rope(**kw):
    return make(E.UspRopeDesc, dict(bs=2, L=8, q_stride=0, q_out_stride=0, k_stride=0, k_out_stride=0, max_pos=8, hq=4, hkv=2,
                                    hd=64, rot=64, dtype=E.USP_BF16, interleaved=0, inverse=0, nseq=0), kw)


def append(**kw):
    return make(E.UspRopeAppendDesc, dict(tokens=4, q_stride=0, q_out_stride=0, k_stride=0, v_stride=0, max_pos=8, nreq=2, hq=4,
                                          rot=64, interleaved=0, dtype=E.USP_BF16), kw)


def cache(**kw):
    return make(E.UspCacheDims, dict(num_pages=8, k_page_stride=0, v_page_stride=0, page_size=16, hkv=2, hd=64,
                                     dtype=E.USP_BF16), kw)


def q4(**kw):
    return make(E.UspQ4Dims, dict(num_pages=8, k_page_stride=0, v_page_stride=0, k_scale_stride=0, v_scale_stride=0,
                                  page_size=16, hkv=2, hd=64), kw)


def attn(cache_kw=None, **kw):
    return make(E.UspPagedQ4Desc, dict(cache=q4(**(cache_kw or {})), tokens=4, q_stride=0, out_stride=0, table_stride=4, nreq=2,
                                       max_pages=4, hq=8, max_new=4, causal=1, scale=0.0, dtype=E.USP_BF16), kw)


ROTATION = [(dict(rot=24), E.USP_ERR_SHAPE), (dict(rot=80), E.USP_ERR_SHAPE), (dict(rot=-16), E.USP_ERR_INVALID_ARG),
            (dict(max_pos=-1), E.USP_ERR_INVALID_ARG), (dict(max_pos=2 ** 31), E.USP_ERR_UNSUPPORTED), (dict(dtype=5), E.USP_ERR_DTYPE),
            (dict(q_stride=8), E.USP_ERR_SHAPE), (dict(q_out_stride=-8), E.USP_ERR_INVALID_ARG), (dict(k_stride=260), E.USP_ERR_ALIGN),
            (dict(q_stride=2 ** 40), E.USP_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", ROTATION + [
    (dict(rot=0), E.USP_ERR_SHAPE), (dict(hq=0), E.USP_ERR_INVALID_ARG), (dict(hkv=-1), E.USP_ERR_INVALID_ARG),
    (dict(hd=96), E.USP_ERR_UNSUPPORTED), (dict(L=-1), E.USP_ERR_INVALID_ARG),
    (dict(bs=2 ** 40), E.USP_ERR_UNSUPPORTED), (dict(bs=2 ** 26), E.USP_ERR_UNSUPPORTED),
    (dict(L=2 ** 31 - 1, max_pos=2 ** 31 - 1), E.USP_ERR_UNSUPPORTED), (dict(nseq=-1), E.USP_ERR_INVALID_ARG),
    (dict(nseq=2 ** 31 - 1), E.USP_ERR_UNSUPPORTED)])
def test_rope_rejects(kw, code):
    assert _abi.load().usp_rope(*([GOOD] * 7), rope(**kw), None) == code


def test_rope_rejects_pointers():
    f, seven = _abi.load().usp_rope, [GOOD] * 7
    for i in range(7):
        if i < 5:
            assert f(*seven[:i], None, *seven[i + 1:], rope(), None) == E.USP_ERR_INVALID_ARG
        assert f(*seven[:i], BAD, *seven[i + 1:], rope(), None) == E.USP_ERR_ALIGN
    assert f(*seven[:5], None, None, rope(nseq=3), None) == E.USP_ERR_INVALID_ARG
    assert f(*seven[:5], None, None, rope(L=9), None) == E.USP_ERR_SHAPE     # more tokens than the table has rows
    assert f(*([None] * 7), rope(bs=0), None) == E.USP_OK
    assert f(*([None] * 7), rope(L=0), None) == E.USP_OK


@pytest.mark.parametrize("kw,code", ROTATION + [
    (dict(tokens=-1), E.USP_ERR_INVALID_ARG), (dict(hq=-1), E.USP_ERR_INVALID_ARG), (dict(nreq=-1), E.USP_ERR_INVALID_ARG),
    (dict(rot=0), E.USP_ERR_SHAPE), (dict(v_stride=64), E.USP_ERR_SHAPE), (dict(tokens=2 ** 28), E.USP_ERR_UNSUPPORTED),
    (dict(nreq=2 ** 30 + 1), E.USP_ERR_UNSUPPORTED)])
def test_rope_append_rejects(kw, code):
    lib = _abi.load()
    assert lib.usp_rope_append(*([GOOD] * 11), append(**kw), cache(), None) == code
    assert lib.usp_rope_append_q4(*([GOOD] * 13), append(**kw), q4(), None) == code


def test_rope_append_rejects_pointers_and_caches():
    lib = _abi.load()
    f, n = lib.usp_rope_append, [GOOD] * 11
    # q, q_out, k, v, k_cache, v_cache, slot_map, positions, cu_new, kv_lens, table
    for i in range(11):
        assert f(*n[:i], BAD, *n[i + 1:], append(), cache(), None) == E.USP_ERR_ALIGN
        if i not in (7, 8, 9):
            assert f(*n[:i], None, *n[i + 1:], append(), cache(), None) == E.USP_ERR_INVALID_ARG
    for i in (8, 9):
        m = n[:7] + [None] + n[8:]
        assert f(*m[:i], None, *m[i + 1:], append(), cache(), None) == E.USP_ERR_INVALID_ARG
    assert f(*n, append(), cache(dtype=E.USP_F32), None) == E.USP_ERR_DTYPE
    assert f(*n, append(), cache(page_size=24), None) == E.USP_ERR_UNSUPPORTED
    assert f(*([None] * 11), append(tokens=0), cache(), None) == E.USP_OK
    g, n = lib.usp_rope_append_q4, [GOOD] * 13
    for i in range(13):
        assert g(*n[:i], BAD, *n[i + 1:], append(), q4(), None) == E.USP_ERR_ALIGN
        if i not in (9, 10, 11):
            assert g(*n[:i], None, *n[i + 1:], append(), q4(), None) == E.USP_ERR_INVALID_ARG


Q4_BAD = [(dict(hd=96), E.USP_ERR_UNSUPPORTED), (dict(hkv=0), E.USP_ERR_INVALID_ARG), (dict(num_pages=-1), E.USP_ERR_INVALID_ARG),
          (dict(page_size=8), E.USP_ERR_UNSUPPORTED), (dict(page_size=48), E.USP_ERR_UNSUPPORTED),
          (dict(num_pages=2 ** 27), E.USP_ERR_UNSUPPORTED), (dict(k_page_stride=1008), E.USP_ERR_SHAPE),
          (dict(v_page_stride=-16), E.USP_ERR_INVALID_ARG), (dict(k_page_stride=1032), E.USP_ERR_ALIGN),
          (dict(k_scale_stride=48), E.USP_ERR_SHAPE), (dict(v_scale_stride=72), E.USP_ERR_ALIGN),
          (dict(v_scale_stride=2 ** 40), E.USP_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", Q4_BAD)
def test_q4_caches_are_checked(kw, code):
    lib = _abi.load()
    assert lib.usp_cache_append_q4(*([GOOD] * 7), 4, 0, 0, E.USP_BF16, q4(**kw), None) == code
    assert lib.usp_rope_append_q4(*([GOOD] * 13), append(), q4(**kw), None) == code
    assert lib.usp_paged_attn_q4(*([GOOD] * 10), attn(kw), GOOD, 2 ** 30, None) == code
    assert lib.usp_paged_attn_q4_workspace_size(attn(kw)) == 0


def test_append_q4_rejects():
    f, n = _abi.load().usp_cache_append_q4, [GOOD] * 7
    for i in range(7):
        assert f(*n[:i], None, *n[i + 1:], 4, 0, 0, E.USP_F32, q4(), None) == E.USP_ERR_INVALID_ARG
        assert f(*n[:i], BAD, *n[i + 1:], 4, 0, 0, E.USP_F32, q4(), None) == E.USP_ERR_ALIGN
    assert f(*n, -1, 0, 0, E.USP_F32, q4(), None) == E.USP_ERR_INVALID_ARG
    assert f(*n, 4, 0, 0, 3, q4(), None) == E.USP_ERR_DTYPE
    assert f(*n, 4, 64, 0, E.USP_F32, q4(), None) == E.USP_ERR_SHAPE
    assert f(*n, 4, 0, 130, E.USP_F32, q4(), None) == E.USP_ERR_ALIGN
    assert f(*n, 2 ** 30, 0, 0, E.USP_F32, q4(), None) == E.USP_ERR_UNSUPPORTED
    assert f(*([None] * 7), 0, 0, 0, E.USP_F32, q4(), None) == E.USP_OK


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), E.USP_ERR_INVALID_ARG), (dict(nreq=-1), E.USP_ERR_INVALID_ARG), (dict(max_new=-1), E.USP_ERR_INVALID_ARG),
    (dict(hq=0), E.USP_ERR_INVALID_ARG), (dict(scale=float("inf")), E.USP_ERR_INVALID_ARG), (dict(scale=float("nan")), E.USP_ERR_INVALID_ARG),
    (dict(hq=7), E.USP_ERR_SHAPE), (dict(table_stride=3), E.USP_ERR_SHAPE), (dict(q_stride=500), E.USP_ERR_SHAPE),
    (dict(out_stride=516), E.USP_ERR_ALIGN), (dict(hq=258), E.USP_ERR_UNSUPPORTED), (dict(tokens=2 ** 28), E.USP_ERR_UNSUPPORTED),
    (dict(dtype=9), E.USP_ERR_DTYPE), (dict(nreq=2 ** 30 + 1), E.USP_ERR_UNSUPPORTED), (dict(q_stride=2 ** 62), E.USP_ERR_UNSUPPORTED)])
def test_attention_rejects(kw, code):
    lib = _abi.load()
    assert lib.usp_paged_attn_q4(*([GOOD] * 10), attn(**kw), GOOD, 2 ** 30, None) == code
    assert lib.usp_paged_attn_q4_workspace_size(attn(**kw)) == 0


def test_attention_rejects_pointers_and_workspace():
    f, n = _abi.load().usp_paged_attn_q4, [GOOD] * 10
    for i in range(10):
        assert f(*n[:i], None, *n[i + 1:], attn(), GOOD, 2 ** 30, None) == E.USP_ERR_INVALID_ARG
        assert f(*n[:i], BAD, *n[i + 1:], attn(), GOOD, 2 ** 30, None) == E.USP_ERR_ALIGN
    assert f(*n, attn(), None, 2 ** 30, None) == E.USP_ERR_INVALID_ARG
    assert f(*n, attn(), GOOD + 128, 2 ** 30, None) == E.USP_ERR_ALIGN
    assert f(*n, attn(dict(num_pages=0)), GOOD, 2 ** 30, None) == E.USP_ERR_SHAPE
    assert f(*([None] * 10), attn(tokens=0), None, 0, None) == E.USP_OK
    assert f(*([None] * 10), attn(nreq=0), None, 0, None) == E.USP_OK


def test_binding_rejects():
    i, t = torch.zeros(3, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    q, c, s = torch.zeros(4, 4, 64), torch.zeros(8, 2, 16, 32, dtype=torch.uint8), torch.zeros(8, 2, 16, 2, dtype=torch.uint8)
    rope_t = torch.zeros(9, 64)
    with pytest.raises(ValueError, match="CUDA"):
        usp.usp_paged_attn_q4(q, c, c, s, s, t, i, i[:2])
    with pytest.raises(ValueError, match="uint8"):
        usp.usp_paged_attn_q4(q, c.float(), c.float(), s, s, t, i, i[:2])
    with pytest.raises(ValueError, match="hd / 32"):
        usp.usp_paged_attn_q4(q, c, c, c, c, t, i, i[:2])
    with pytest.raises(ValueError, match="head dim"):
        usp.usp_paged_attn_q4(torch.zeros(4, 4, 128), c, c, s, s, t, i, i[:2])
    with pytest.raises(ValueError, match="CUDA"):
        usp.usp_cache_append_q4(q[:, :2], q[:, :2], c, c, s, s, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="like the cache"):
        usp.usp_cache_append_q4(q, q, c, c, s, s, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        usp.usp_rope(q[None], q[None], rope_t)
    with pytest.raises(ValueError, match="fp32"):
        usp.usp_rope(q[None], q[None], rope_t.double())
    with pytest.raises(ValueError, match="bs, L"):
        usp.usp_rope(q, q, rope_t)
    with pytest.raises(ValueError, match="4-bit"):
        usp.usp_rope_append(None, q[:, :2], q[:, :2], c, c, torch.zeros(4, dtype=torch.int32), rope_t, i, i[:2])
