"""GPU: rows entering the 8-bit cache, code for code against the oracle."""
import numpy as np
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import K8, KV8Case

pytestmark = pytest.mark.gpu


def state(case):
    return [t.cpu().numpy().copy() for t in (case.k.view(torch.uint8), case.k_scale, case.v.view(torch.uint8), case.v_scale)]


def expect(case, before, starts, n, kn, vn, requests):
    kc, ks, vc, vs = (a.copy() for a in before)
    for r in requests:
        K8.append_request(kc, ks, case.pt[r], int(starts[r]), kn[r, : n[r]].float().cpu().numpy())
        K8.append_request(vc, vs, case.pt[r], int(starts[r]), vn[r, : n[r]].float().cpu().numpy())
    return kc, ks, vc, vs


def assert_state(case, want):
    for got, w, what in zip(state(case), want, ("k", "k_scale", "v", "v_scale")):
        np.testing.assert_array_equal(got, w, err_msg=what)


def rows(case, T, seed, spread=6):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (case.nr, T, case.Hkv, case.d)
    mag = lambda: torch.exp2(torch.randint(-spread, spread, (case.nr, T, case.Hkv, 1), generator=g, device="cuda").float())  # noqa: E731
    return [(torch.randn(shape, generator=g, device="cuda") * mag()).to(torch.bfloat16) for _ in range(2)]


@pytest.mark.parametrize("Hkv,d,lens,T", [
    (8, 128, [0, 1, 15, 16, 17, 31, 200], 7),      # a round's rows at every kind of offset
    (8, 128, [0, 5, 16], 1),                       # a draft step's row
    (1, 64, [0, 9, 100], 33),
    (3, 64, [7, 0], 16),                           # heads that do not fill a CTA
    (5, 128, [2, 14], 100),
])
@pytest.mark.parametrize("ragged", [False, True])
def test_append_matches_oracle(Hkv, d, lens, T, ragged):
    case = KV8Case(Hkv, d, lens, T, seed=T + sum(lens), upto=0).cuda(Hkv)
    n = np.random.default_rng(T).integers(0, T + 1, size=case.nr) if ragged else np.full(case.nr, T)
    kn, vn = rows(case, T, seed=1)
    before = state(case)
    s3r.s3r_kv8_append(case.cache, case.batch, kn, vn, case.ws,
                       n_new=torch.as_tensor(n.astype(np.int32)).cuda() if ragged else None)
    assert s3r.s3r_get_error(case.ws) == 0
    want = expect(case, before, case.lens, n, kn, vn, range(case.nr))
    assert_state(case, want)
    s3r.s3r_kv8_append(case.cache, case.batch, kn, vn, case.ws,
                       n_new=torch.as_tensor(n.astype(np.int32)).cuda() if ragged else None)
    assert_state(case, want)   # the same rows again change nothing


def test_append_offsets_strides_subset_and_foreign_scales():
    """Steps of a longer block in place (a strided view at an offset), for a shuffled subset, over
    pages whose scales are no powers of two."""
    lens = [3, 30, 16, 77]
    case = KV8Case(2, 128, lens, 8, seed=5, pow2=False, upto=0).cuda(2)
    kb, vb = rows(case, 6, seed=2)
    ids = [3, 0, 2]
    batch = s3r.make_batch(case.seq_lens, case.page_table, req_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))
    for i in range(6):
        before = state(case)
        first = np.array([i, i, i, i], dtype=np.int32)
        s3r.s3r_kv8_append(case.cache, batch, kb[:, i:i + 1], vb[:, i:i + 1], case.ws, first=torch.as_tensor(first).cuda())
        assert s3r.s3r_get_error(case.ws) == 0
        assert_state(case, expect(case, before, case.lens + first, np.ones(4, int), kb[:, i:i + 1], vb[:, i:i + 1], ids))


def test_append_extreme_values():
    """Zeros, the largest and smallest bf16, exact borders of a scale, and non-finite elements."""
    case = KV8Case(1, 64, [0, 0, 0, 0, 0, 0, 0, 0], 2, seed=1, upto=0).cuda(1)
    kn, vn = (torch.zeros((8, 2, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    top = torch.finfo(torch.bfloat16)
    for r, x in enumerate((0.0, top.max, 1e-40, 448.0, 450.0, 1.75, 1.7578125, top.tiny)):
        kn[r, 0, 0, 3], vn[r, 1, 0, 63] = x, -x
    before = state(case)
    s3r.s3r_kv8_append(case.cache, case.batch, kn, vn, case.ws)
    assert s3r.s3r_get_error(case.ws) == 0
    assert_state(case, expect(case, before, case.lens, [2] * 8, kn, vn, range(8)))
    kn[2, 1, 0, 5], kn[4, 0, 0, 0], vn[6, 0, 0, 1] = float("nan"), float("inf"), -float("inf")
    before = state(case)
    s3r.s3r_kv8_append(case.cache, case.batch, kn, vn, case.ws)
    assert s3r.s3r_get_error(case.ws) == 1 << 6
    assert_state(case, expect(case, before, case.lens, [2] * 8, kn, vn, range(8)))


def test_append_reports_and_skips_what_does_not_fit():
    case = KV8Case(2, 64, [10, 20, 30, 40], 8, seed=9, upto=0).cuda(2)
    kn, vn = rows(case, 4, seed=3)
    case.page_table[1, 1] = case.total        # request 1: its second page's id is outside the pool
    n = np.array([4, 4, 5, -1], dtype=np.int32)   # request 2, 3: more rows than given, fewer than none
    before = state(case)
    s3r.s3r_kv8_append(case.cache, case.batch, kn, vn, case.ws, n_new=torch.as_tensor(n).cuda())
    assert s3r.s3r_get_error(case.ws) == 1 << 5
    assert_state(case, expect(case, before, case.lens, [4, 0, 0, 0], kn, vn, [0]))
    first = np.array([0, -1, case.max_pages * 16 - 33, 2], dtype=np.int32)   # 2: past the capacity
    before = state(case)
    s3r.s3r_kv8_append(case.cache, case.batch, kn, vn, case.ws, first=torch.as_tensor(first).cuda())
    # request 3's kept rows 40 and 41 were never written and hold NaN codes: zeros now, and reported
    assert s3r.s3r_get_error(case.ws) == (1 << 5) | (1 << 6)
    assert_state(case, expect(case, before, case.lens + first, [4, 0, 0, 4], kn, vn, [0, 3]))


def test_binding_refuses_wrong_tensors():
    case = KV8Case(2, 64, [10, 20], 8, seed=9, upto=0).cuda(4)
    kn, vn = rows(case, 4, seed=3)
    before = state(case)
    for bad in (lambda: s3r.s3r_kv8_append(case.cache, case.batch, kn[:1], vn[:1], case.ws),
                lambda: s3r.s3r_kv8_append(case.cache, case.batch, kn, vn.cpu(), case.ws),
                lambda: s3r.s3r_kv8_append(case.cache, case.batch, kn.float(), vn.float(), case.ws),
                lambda: s3r.s3r_kv8_append(case.cache, case.batch, kn, vn[:, :2], case.ws),
                lambda: s3r.s3r_kv8_append(case.cache, case.batch, kn.transpose(1, 2), vn.transpose(1, 2), case.ws),
                lambda: s3r.s3r_kv8_append(case.cache, case.batch, kn, vn, case.ws, n_new=torch.ones(2, device="cuda")),
                lambda: s3r.s3r_kv8_append(case.cache, s3r.make_batch(case.seq_lens), kn, vn, case.ws),
                lambda: s3r.make_kv8_cache(case.k, case.v, case.k_scale[:, :1], case.v_scale, 4),
                lambda: s3r.make_kv8_cache(case.k.float(), case.v, case.k_scale, case.v_scale, 4)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    assert_state(case, before)
