"""GPU: pages, scales and scores that lie past 32-bit offsets give what the same ones give near the start."""
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import KV8Case
from tests.test_gpu_kv8_append import rows
from tests.test_gpu_kv8_attention import draft_sets, run_draft, run_verify

pytestmark = pytest.mark.gpu


def test_pages_past_32_bit_offsets():
    """A pool of 5.4 GB per tensor whose used pages are its last: append, verify and draft bit for bit as over
    the small pool; nothing else of the large one changes."""
    case = KV8Case(8, 128, [3000, 777, 16], 8, seed=41).cuda(32, sel_stride=3100)
    far = KV8Case(8, 128, [3000, 777, 16], 8, seed=41)
    total = 330_000
    base = total - far.total
    assert base * 8 * 16 * 128 > 1 << 32
    idx, n = draft_sets(case, [900, 700, 16], seed=1)
    near = [case.k, case.v, case.k_scale, case.v_scale]
    big = [torch.zeros((total, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in near]
    for b, t in zip(big, near):
        b[base:] = t
    far.k, far.v, far.k_scale, far.v_scale = big
    far.seq_lens = case.seq_lens
    far.page_table = torch.where(case.page_table >= 0, case.page_table + base, case.page_table)
    far.cache, far.batch = s3r.make_kv8_cache(*big, 32), s3r.make_batch(far.seq_lens, far.page_table)
    far.ws = s3r.new_workspace(s3r.s3r_kv8_workspace_size(far.cache, 3, far.max_pages, 8, 64, 3100))
    kn, vn = rows(case, 7, seed=2)
    got = []
    for c in (case, far):
        s3r.s3r_kv8_append(c.cache, c.batch, kn, vn, c.ws)
        got.append([*run_verify(c, 32, 6, seed=3)[1:], *run_draft(c, 32, [5, 0, 6], idx, n, seed=4)[1:]])
        assert s3r.s3r_get_error(c.ws) == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
    for b, t in zip(big, near):
        assert torch.equal(b[base:], t) and not b[:base].any()


def test_scores_past_32_bit_offsets():
    """64 rows of scores over a capacity of 2^23 positions and 8 heads: the last row starts at 16 GB."""
    case = KV8Case(8, 128, [2000], 8, seed=43).cuda(64)
    q, out, lse, sc = run_verify(case, 64, 7, seed=5)
    cap = 1 << 23
    wide = torch.full((1, cap // 16), -1, dtype=torch.int32, device="cuda")
    wide[:, : case.max_pages] = case.page_table
    batch = s3r.make_batch(case.seq_lens, wide)
    ws = s3r.new_workspace(s3r.s3r_kv8_workspace_size(case.cache, 1, cap // 16, 7, 64, 1))
    big = torch.empty((1, 8, 64, cap), device="cuda")
    big[..., 1900:2100] = 7.0
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    s3r.s3r_verify_attn_kv8(case.cache, batch, 7, q, out2, lse2, big, ws)
    assert s3r.s3r_get_error(ws) == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert torch.equal(big[..., :2000], sc[..., :2000]) and (big[..., 2000:2100] == 7.0).all()
