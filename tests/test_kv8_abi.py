"""CPU checks of the 8-bit cache's and the page calls' entry points: sizes and refusals on the host
(nothing is launched without a GPU)."""
import ctypes

import pytest

OK, ARG, UNSUPPORTED, WS = 0, 1, 2, 4


def _cache(k_scale=0x3000, v_scale=0x4000, **kw):
    import sparse_dense_kv_b200 as s3r
    d = dict(num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16, num_pages=1000, k_pool=0x100000, v_pool=0x200000)
    d.update(kw)
    return s3r.KV8CacheDesc(s3r.KVCacheDesc(**d), k_scale, v_scale)


def _batch(**kw):
    import sparse_dense_kv_b200 as s3r
    d = dict(batch=4, num_requests=4, req_ids=None, seq_lens=0x1000, page_table=0x2000, max_pages_per_req=100)
    d.update(kw)
    return s3r.BatchDesc(**d)


def test_workspace_sizes():
    import sparse_dense_kv_b200 as s3r
    c = _cache()
    a = s3r.s3r_kv8_workspace_size(c, 32, 1540, 6, 151936, 1232)
    assert 0 < a <= s3r.s3r_kv8_workspace_size(c, 64, 1540, 6, 151936, 1232)
    assert a <= s3r.s3r_kv8_workspace_size(c, 32, 1540, 8, 151936, 1232)
    assert a <= s3r.s3r_kv8_workspace_size(c, 32, 1540, 6, 151936, 100000)
    for bad in (_cache(head_dim=96), _cache(k_scale=None), _cache(v_scale=0x4002), _cache(page_size=32)):
        with pytest.raises(s3r.S3RError):
            s3r.s3r_kv8_workspace_size(bad, 32, 1540, 6, 64, 64)
    assert s3r.s3r_pages_workspace_size(0) > 0
    with pytest.raises(s3r.S3RError):
        s3r.s3r_pages_workspace_size(-1)


def test_attention_refusals():
    import sparse_dense_kv_b200 as s3r
    L, ref = s3r.lib, ctypes.byref
    big = 1 << 34

    def verify(c=None, b=None, k=6, q=0x10, out=0x20, lse=0x30, sc=None, ws=0x100, n=big):
        return L.s3r_verify_attn_kv8(ref(c or _cache()), ref(b or _batch()), k, q, out, lse, sc, ws, n, None)

    def draft(c=None, b=None, step=0x10, q=0x20, qs=0, idx=0x30, stride=64, cnt=0x40, out=0x50, lse=None, ws=0x100, n=big):
        return L.s3r_sparse_draft_attn_kv8(ref(c or _cache()), ref(b or _batch()), step, q, qs, idx, stride, cnt, out, lse, ws, n, None)

    assert L.s3r_verify_attn_kv8(None, None, 6, 0x10, 0x10, 0x10, None, 0x100, big, None) == ARG
    for call in (verify, draft):
        assert call(b=_batch(batch=0)) == OK
        assert call(c=_cache(head_dim=96)) == UNSUPPORTED
        assert call(c=_cache(page_size=32)) == UNSUPPORTED
        assert call(c=_cache(num_q_heads=72)) == UNSUPPORTED       # 9 query heads per KV head
        assert call(c=_cache(num_q_heads=33)) == ARG
        assert call(c=_cache(k_pool=0x100008)) == ARG
        assert call(c=_cache(k_scale=None)) == ARG
        assert call(c=_cache(v_scale=0x4001)) == ARG
        assert call(c=_cache(num_pages=1 << 25)) == UNSUPPORTED    # rows past 31 bits
        assert call(b=_batch(page_table=None)) == ARG
        assert call(b=_batch(seq_lens=None)) == ARG
        assert call(b=_batch(batch=5)) == ARG
        assert call(b=_batch(batch=70000, num_requests=70000)) == UNSUPPORTED
        assert call(b=_batch(max_pages_per_req=1 << 27)) == UNSUPPORTED
        assert call(q=None) == ARG and call(q=0x18) == ARG and call(out=0x58) == ARG
        assert call(ws=None) == WS and call(ws=0x180) == WS and call(n=4096) == WS
    assert verify(k=9) == UNSUPPORTED and verify(k=-1) == UNSUPPORTED
    assert verify(c=_cache(num_q_heads=64), k=8) == UNSUPPORTED     # 72 rows
    assert verify(sc=0x18) == ARG and verify(lse=0x31) == ARG and verify(lse=None) == ARG
    assert draft(qs=100) == ARG and draft(qs=32 * 128 + 4) == ARG and draft(stride=0) == ARG
    assert draft(step=None) == ARG and draft(idx=0x31) == ARG and draft(cnt=None) == ARG and draft(lse=0x52) == ARG


def test_append_refusals():
    import sparse_dense_kv_b200 as s3r

    def append(c=None, b=None, first=None, T=7, n_new=None, k=0x10, v=0x20, stride=0, ws=0x100, n=1 << 20):
        return s3r.lib.s3r_kv8_append(ctypes.byref(c or _cache()), ctypes.byref(b or _batch()), first, T, n_new, k, v, stride, ws, n, None)

    assert append(T=0) == OK and append(b=_batch(batch=0)) == OK
    assert append(T=-1) == ARG and append(T=1 << 30) == ARG and append(k=None) == ARG and append(v=0x24) == ARG
    assert append(first=0x11) == ARG and append(n_new=0x12) == ARG
    assert append(stride=7 * 8 * 128 - 8) == ARG and append(stride=7 * 8 * 128 + 4) == ARG
    assert append(c=_cache(k_scale=None)) == ARG and append(ws=None) == WS and append(n=8) == WS


def test_page_refusals():
    import sparse_dense_kv_b200 as s3r

    def alloc(b=None, pt=0x10, T=7, n_new=None, held=0x10, free=0x10, count=0x10, cap=100, ho=0x10, co=0x10, granted=0x10, slots=None,
              ws=0x100, n=1 << 20):
        return s3r.lib.s3r_alloc_pages(ctypes.byref(b or _batch()), pt, T, n_new, held, free, count, cap, ho, co, granted, slots, ws, n, None)

    def release(b=None, pt=0x10, keep=None, held=0x10, free=0x10, count=0x10, cap=100, ho=0x10, co=0x10, ws=0x100, n=1 << 20):
        return s3r.lib.s3r_release_pages(ctypes.byref(b or _batch()), pt, keep, held, free, count, cap, ho, co, ws, n, None)

    for call in (alloc, release):
        assert call(b=_batch(batch=0)) == OK
        for name in ("pt", "held", "free", "count", "ho", "co"):
            assert call(**{name: None}) == ARG and call(**{name: 0x12}) == ARG
        assert call(cap=-1) == ARG and call(b=_batch(max_pages_per_req=0)) == ARG
        assert call(b=_batch(batch=5)) == ARG and call(b=_batch(batch=70000, num_requests=70000)) == UNSUPPORTED
        assert call(ws=None) == WS and call(ws=0x101) == WS and call(n=64) == WS
    assert alloc(T=-1) == ARG and alloc(granted=None) == ARG and alloc(slots=0x14) == ARG and alloc(n_new=0x11) == ARG
    assert release(keep=0x13) == ARG
