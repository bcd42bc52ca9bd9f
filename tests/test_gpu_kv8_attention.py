"""GPU parity of the 8-bit cache's verify and sparse draft attention against 64-bit attention."""
import numpy as np
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import DRAFT, VERIFY, KV8Case, assert_within, attention_bounds, f64, rows_of

pytestmark = pytest.mark.gpu


def run_verify(case, Hq, k, seed, scores=True, q=None):
    T, G = k + 1, Hq // case.Hkv
    g = torch.Generator(device="cuda").manual_seed(seed)
    if q is None:
        q = torch.randn((case.nr, T, Hq, case.d), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, float("nan"))
    lse = torch.full((case.nr, T, Hq), float("nan"), device="cuda")
    sc = torch.full((case.nr, case.Hkv, G * T, case.max_pages * 16), 7.0, device="cuda") if scores else None
    s3r.s3r_verify_attn_kv8(case.cache, case.batch, k, q, out, lse, sc, case.ws)
    return q, out, lse, sc


def check_verify(case, Hq, k, q, out, lse, sc, requests=None):
    T, G = k + 1, Hq // case.Hkv
    for r in range(case.nr) if requests is None else requests:
        L = int(case.lens[r])
        K, V = case.values(r, L + T)
        vis = np.arange(L + T)[None, :] <= L + (np.arange(G * T) // G)[:, None]
        o, l, x, bo, bl, bx = attention_bounds(rows_of(f64(q[r]), case.Hkv), K, V, vis, **VERIFY)
        got = rows_of(f64(out[r]), case.Hkv)
        assert_within(got, o, bo, f"out r={r} L={L}")
        assert_within(rows_of(f64(lse[r])[..., None], case.Hkv)[..., 0], l, bl, f"lse r={r} L={L}")
        if sc is not None:
            assert_within(f64(sc[r])[:, :, :L], x[:, :, :L], bx[:, :, :L] + 1e-30, f"scores r={r} L={L}")
            assert (sc[r][:, :, L:] == 7.0).all()   # nothing is written past L


@pytest.mark.parametrize("Hq,Hkv,d,k,lens", [
    (2, 1, 64, 6, [256, 300]),                       # the tests' tiny workload
    (16, 8, 128, 0, [77]),                           # one row, one tile
    (16, 8, 128, 0, [0, 1, 15, 16, 17, 127, 128]),   # one row, shortest contexts
    (8, 1, 128, 2, [5, 17, 0, 33]),                  # G = 8, block as long as the context
    (32, 8, 128, 6, [1000, 2049, 3071, 64]),         # 28 rows (32 wide)
    (32, 8, 128, 8, [1030, 2000, 121, 120]),         # 36 rows (48 wide), block across a tile's edge
    (64, 8, 128, 5, [700, 127, 129]),                # 48 rows, no padding
    (64, 8, 128, 7, [1500, 900, 769]),               # 64 rows
    (12, 4, 64, 4, [333, 1200]),                     # G = 3, d = 64, 15 rows
    (64, 8, 64, 7, [333, 1200]),                     # 64 rows, d = 64
    (40, 8, 64, 7, [333, 1200]),                     # 40 rows, d = 64
    (4, 4, 128, 3, [65, 1023]),                      # G = 1
    (32, 8, 128, 6, [9000, 12000, 7000, 10000, 30000]),   # several chunks per span
])
def test_verify_matches_64_bit(Hq, Hkv, d, k, lens):
    case = KV8Case(Hkv, d, lens, k + 1, seed=sum(lens) + k).cuda(Hq)
    res = run_verify(case, Hq, k, seed=5)
    assert s3r.s3r_get_error(case.ws) == 0
    check_verify(case, Hq, k, *res)


def test_verify_any_scale_and_large_and_small_values():
    """Scales that are no powers of two and differ by 2^24 from page to page; q rows of very
    different magnitude, one all zero."""
    case = KV8Case(2, 128, [700, 130, 1], 3, seed=3, pow2=False, scale_spread=24).cuda(8)
    q = torch.randn((3, 3, 8, 128), device="cuda") * torch.exp2(torch.arange(8, device="cuda").float() * 3 - 12)[None, None, :, None]
    q[1, 1, 3] = 0
    res = run_verify(case, 8, 2, seed=9, q=q.to(torch.bfloat16))
    assert s3r.s3r_get_error(case.ws) == 0
    check_verify(case, 8, 2, *res)


def test_verify_v_scales_that_grow_along_a_span():
    """Runs of four tiles (a chunk) with V scales of 2^-119 before a tile of ordinary ones, several
    chunks to a span; one page far above; scales above 2^48 are reported and taken as that."""
    case = KV8Case(8, 128, [9000, 12000, 7000, 10000, 30000], 7, seed=23).cuda(32)
    for r in range(case.nr):
        pages = [int(x) for i, x in enumerate(case.pt[r]) if x >= 0 and i // 8 % 5 < 4]
        case.v_scale[torch.tensor(pages, device="cuda")] = 2.0 ** -119
    case.v_scale[int(case.pt[2, 120]), 1] = 2.0 ** 40
    case.v_scale[int(case.pt[1, 3])] = 2.0 ** -100
    res = run_verify(case, 32, 6, seed=11, scores=False)
    assert s3r.s3r_get_error(case.ws) == 0
    check_verify(case, 32, 6, *res)
    case.v_scale[int(case.pt[1, 7]), 0] = 2.0 ** 60
    res = run_verify(case, 32, 6, seed=11, scores=False)
    assert s3r.s3r_get_error(case.ws) == 1 << 6
    case.v_scale[int(case.pt[1, 7]), 0] = 2.0 ** 48
    check_verify(case, 32, 6, *res)


def test_verify_one_dominant_position_and_constant_values():
    """A key far above the rest (its weight 1, the others' 2^-18 each) and values of one sign, so
    that small weights' roundings would add up."""
    case = KV8Case(1, 128, [2000], 1, seed=4, std=0.0).cuda(1)
    case.v.copy_(torch.full_like(case.v, 0x38))          # 1.0
    case.v_scale.fill_(1.0)
    case.k_scale.fill_(1.0)
    pg = case.pt[0, 37]
    case.k[pg, 0, 5] = 0x38
    q = torch.full((1, 1, 1, 128), 12.5 / 128 ** 0.5, device="cuda").to(torch.bfloat16)
    res = run_verify(case, 1, 0, seed=1, q=q)
    check_verify(case, 1, 0, *res)


def test_verify_without_capture_is_the_same_and_repeats_bit_for_bit():
    case = KV8Case(8, 128, [5000, 333, 1024], 7, seed=8).cuda(32)
    q, o1, l1, s1 = run_verify(case, 32, 6, seed=2)
    for scores in (False, True, False):
        _, o2, l2, s2 = run_verify(case, 32, 6, seed=2, scores=scores)
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
        assert s2 is None or torch.equal(s1, s2)


def test_verify_subset_and_bad_requests():
    """A shuffled subset: others' outputs stay untouched; an id out of range, a context past the
    page table and a negative length are reported and skipped."""
    lens = [500, 40, 900, 10, 260]
    case = KV8Case(2, 128, lens, 2, seed=6).cuda(4)
    for ids, bad in (([3, 0, 4], ()), ([2, 5, 1], ()), ([2, -1, 1], ()), ([0, 1, 2, 3], (1, 3))):
        lens_t = case.seq_lens.clone()
        if bad:
            lens_t[1], lens_t[3] = case.max_pages * 16, -4
        batch = s3r.make_batch(lens_t, case.page_table, req_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))
        q = torch.randn((5, 2, 4, 128), device="cuda").to(torch.bfloat16)
        out, lse = torch.full_like(q, 3.0), torch.full((5, 2, 4), 3.0, device="cuda")
        s3r.s3r_verify_attn_kv8(case.cache, batch, 1, q, out, lse, None, case.ws)
        err = s3r.s3r_get_error(case.ws)
        good = [i for i in ids if 0 <= i < 5 and i not in bad]
        assert err == (0 if len(good) == len(ids) else 1 << 5)
        check_verify(case, 4, 1, q, out, lse, None, requests=good)
        for r in set(range(5)) - set(good):
            assert (out[r] == 3.0).all() and (lse[r] == 3.0).all()


def test_verify_bad_page_reads_as_zero_rows():
    """A page id outside the pool: reported, its rows count as zero keys and values."""
    case = KV8Case(2, 128, [300, 300], 1, seed=7).cuda(4)
    case.page_table[1, 3] = case.total
    case.page_table[1, 7] = -1
    q, out, lse, sc = run_verify(case, 4, 0, seed=3)
    assert s3r.s3r_get_error(case.ws) == 1 << 5
    check_verify(case, 4, 0, q, out, lse, sc, requests=[0])
    K, V = case.values(1, 301)
    for pg in (3, 7):
        K[:, pg * 16:(pg + 1) * 16] = 0
        V[:, pg * 16:(pg + 1) * 16] = 0
    o, l, x, bo, bl, bx = attention_bounds(rows_of(f64(q[1]), 2), K, V, np.ones((2, 301), bool), **VERIFY)
    assert_within(rows_of(f64(out[1]), 2), o, bo, "out")
    assert_within(rows_of(f64(lse[1])[..., None], 2)[..., 0], l, bl, "lse")


def test_verify_bad_scales_and_nan_queries():
    case = KV8Case(2, 128, [300, 200], 1, seed=17).cuda(4)
    case.v_scale[case.pt[0, 2], 1] = float("inf")
    case.k_scale[case.pt[0, 4], 0] = float("nan")
    q, out, lse, _ = run_verify(case, 4, 0, seed=3, scores=False)
    assert s3r.s3r_get_error(case.ws) == 1 << 6
    case.v_scale[case.pt[0, 2], 1] = 0
    case.k_scale[case.pt[0, 4], 0] = 0
    check_verify(case, 4, 0, q, out, lse, None)
    q[1, 0, 2, 5] = float("nan")
    q[1, 0, 0, 9] = float("inf")
    _, out2, lse2, _ = run_verify(case, 4, 0, seed=3, scores=False, q=q)
    assert s3r.s3r_get_error(case.ws) == 1 << 6
    assert out2[1, 0, [0, 2]].isnan().all() and lse2[1, 0, [0, 2]].isnan().all()   # their own rows only
    assert torch.equal(out2[1, 0, [1, 3]], out[1, 0, [1, 3]]) and torch.equal(out2[0], out[0])


def test_verify_more_requests_than_one_launch_takes():
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 300, size=300)]
    case = KV8Case(1, 64, lens, 1, seed=21).cuda(2)
    res = run_verify(case, 2, 0, seed=4)
    assert s3r.s3r_get_error(case.ws) == 0
    check_verify(case, 2, 0, *res)


def test_verify_wait_limit_reports_and_recovers():
    """Waits that run out on purpose report S3R_ERR_TIMEOUT; the next launch is right again (the
    workspace re-zeroed: a launch that gave up left its counters as they were)."""
    case = KV8Case(8, 128, [20000] * 8, 7, seed=2).cuda(32)
    s3r.s3r_set_wait_limit(1)
    try:
        run_verify(case, 32, 6, seed=1)
        assert s3r.s3r_get_error(case.ws) & (1 << 7)
    finally:
        s3r.s3r_set_wait_limit(0)
    s3r.s3r_workspace_init(case.ws)
    res = run_verify(case, 32, 6, seed=1)
    assert s3r.s3r_get_error(case.ws) == 0
    check_verify(case, 32, 6, *res, requests=[0, 7])


# ------------------------------------------------------------------------------- draft
def draft_sets(case, sizes, seed):
    """Per (request, head) sorted distinct positions below L, sizes[r] of them (capped at L)."""
    rng = np.random.default_rng(seed)
    n = [min(int(s), int(L)) for s, L in zip(sizes, case.lens)]
    stride = max(1, max(n)) + 3
    idx = np.full((case.nr, case.Hkv, stride), -9, dtype=np.int32)
    for r in range(case.nr):
        for h in range(case.Hkv):
            idx[r, h, : n[r]] = np.sort(rng.choice(int(case.lens[r]), size=n[r], replace=False)) if n[r] else []
    return idx, n


def run_draft(case, Hq, steps, idx, n, seed, batch=None, q=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if q is None:
        q = torch.randn((case.nr, Hq, case.d), generator=g, device="cuda").to(torch.bfloat16)
    out, lse = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((case.nr, Hq), 3.0, device="cuda")
    cnt = torch.as_tensor(np.repeat(np.asarray(n, dtype=np.int32)[:, None], case.Hkv, 1)).cuda()
    s3r.s3r_sparse_draft_attn_kv8(case.cache, batch or case.batch, torch.tensor(steps, dtype=torch.int32, device="cuda"), q,
                                  torch.as_tensor(idx).cuda(), cnt, out, lse, case.ws)
    return q, out, lse


def check_draft(case, Hq, steps, idx, n, q, out, lse, requests=None):
    G = Hq // case.Hkv
    for r in range(case.nr) if requests is None else requests:
        L = int(case.lens[r])
        K, V = case.values(r, L + steps[r] + 1)
        for h in range(case.Hkv):
            at = np.concatenate([idx[r, h, : n[r]], np.arange(L, L + steps[r] + 1)]).astype(np.int64)
            rows = f64(q[r])[h * G:(h + 1) * G][None]
            o, l, _, bo, bl, _ = attention_bounds(rows, K[h: h + 1, at], V[h: h + 1, at], np.ones((G, at.size), bool), **DRAFT)
            assert_within(f64(out[r])[h * G:(h + 1) * G][None], o, bo, f"out r={r} h={h}")
            assert_within(f64(lse[r])[h * G:(h + 1) * G][None], l, bl, f"lse r={r} h={h}")


@pytest.mark.parametrize("Hq,Hkv,d,lens,sizes,steps", [
    (2, 1, 64, [256, 300], [64, 75], [0, 5]),
    (32, 8, 128, [1000, 2049, 3000, 64], [50, 600, 3000, 64], [0, 3, 5, 7]),
    (8, 1, 128, [5, 17, 0, 33, 1], [0, 1, 0, 31, 1], [0, 0, 0, 2, 7]),      # empty and one-position sets
    (16, 8, 128, [200], [127], [0]),                                        # one chunk, exactly
    (12, 4, 64, [400, 400], [127, 128], [0, 0]),                            # at a chunk's edge
    (64, 8, 64, [700], [600], [7]),
    (4, 4, 128, [6000], [6000], [1]),                                       # many chunks
    (6, 2, 128, [31, 32, 33, 95, 96, 97], [31, 32, 33, 95, 96, 97], [0, 0, 0, 0, 0, 0]),
])
def test_draft_matches_64_bit(Hq, Hkv, d, lens, sizes, steps):
    case = KV8Case(Hkv, d, lens, 8, seed=sum(lens)).cuda(Hq, sel_stride=max(lens) + 4)
    idx, n = draft_sets(case, sizes, seed=1)
    res = run_draft(case, Hq, steps, idx, n, seed=5)
    assert s3r.s3r_get_error(case.ws) == 0
    check_draft(case, Hq, steps, idx, n, *res)


def test_draft_any_scale_strided_queries_and_subset():
    case = KV8Case(2, 128, [900, 40, 700], 8, seed=12, pow2=False, scale_spread=24).cuda(8, sel_stride=1000)
    idx, n = draft_sets(case, [300, 40, 650], seed=2)
    block = torch.randn((3, 5, 8, 128), device="cuda").to(torch.bfloat16)
    steps = [2, 2, 2]
    batch = s3r.make_batch(case.seq_lens, case.page_table, req_ids=torch.tensor([2, 0], dtype=torch.int32, device="cuda"))
    res = run_draft(case, 8, steps, idx, n, seed=5, batch=batch, q=block[:, 2])
    assert s3r.s3r_get_error(case.ws) == 0
    check_draft(case, 8, steps, idx, n, *res, requests=[0, 2])
    assert (res[1][1] == 3.0).all() and (res[2][1] == 3.0).all()
    whole = run_draft(case, 8, steps, idx, n, seed=5, q=block[:, 2].contiguous())
    check_draft(case, 8, steps, idx, n, *whole)


def test_draft_bad_inputs_are_reported_and_skipped():
    case = KV8Case(2, 128, [300, 200, 100], 8, seed=13).cuda(4, sel_stride=310)
    idx, n = draft_sets(case, [100, 60, 50], seed=3)
    bad = idx.copy()
    bad[0, 0, 3] = 300          # not below L
    bad[0, 1, 4] = -1
    q, out, lse = run_draft(case, 4, [0, 0, 0], bad, n, seed=1)
    assert s3r.s3r_get_error(case.ws) == 1 << 5
    check_draft(case, 4, [0, 0, 0], idx, n, q, out, lse, requests=[1, 2])
    q, out, lse = run_draft(case, 4, [0, 8, 0], idx, [100, 60, 5000], seed=1)   # step and count out of range
    assert s3r.s3r_get_error(case.ws) == 1 << 5
    check_draft(case, 4, [0, 0, 0], idx, n, q, out, lse, requests=[0])
    assert (out[1:] == 3.0).all()
    q[0, 1, 7] = float("nan")
    _, out2, lse2 = run_draft(case, 4, [0, 0, 0], idx, n, seed=1, q=q)
    assert s3r.s3r_get_error(case.ws) == 1 << 6
    assert out2[0, 1].isnan().all() and lse2[0, 1].isnan() and not out2[0, [0, 2, 3]].isnan().any()
    check_draft(case, 4, [0, 0, 0], idx, n, q, out2, lse2, requests=[1, 2])
