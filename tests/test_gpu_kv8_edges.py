"""GPU: calls at the edges of what the 8-bit cache's documentation allows."""
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import KV8Case
from tests.test_gpu_kv8_append import assert_state, expect, rows, state
from tests.test_gpu_kv8_attention import check_draft, check_verify, draft_sets, run_draft

pytestmark = pytest.mark.gpu


def test_append_of_no_rows_leaves_the_page_alone():
    """A request with n_new = 0 in the middle of a page receives no row: neither codes nor scale of
    that page change (its scale is no power of two and larger than its kept rows need), and a page
    that is not there is not missed. The others' rows enter as ever."""
    case = KV8Case(2, 64, [5, 16, 21, 0, 37], 4, seed=4, pow2=False, upto=0).cuda(2)
    kn, vn = rows(case, 2, seed=3)
    case.page_table[4, 2] = -1
    for n in ([0, 0, 0, 0, 0], [0, 2, 1, 2, 0]):
        before = state(case)
        s3r.s3r_kv8_append(case.cache, case.batch, kn, vn, case.ws, n_new=torch.tensor(n, dtype=torch.int32, device="cuda"))
        assert s3r.s3r_get_error(case.ws) == 0
        assert_state(case, expect(case, before, case.lens, n, kn, vn, range(4)))


def test_draft_over_a_padded_list_of_requests():
    """More ids than requests, those out of range reported and skipped: the real ones, at the list's
    end and in sets of several chunks, use no more of the workspace than without the padding."""
    case = KV8Case(2, 128, [900, 700, 1000, 30], 8, seed=14).cuda(8, sel_stride=1003)
    idx, n = draft_sets(case, [900, 650, 1000, 30], seed=2)
    assert idx.shape[2] == 1003
    guard = torch.full((case.ws.numel() + (1 << 24),), 0x5A, dtype=torch.uint8, device="cuda")
    need = s3r.s3r_kv8_workspace_size(case.cache, 4, case.max_pages, 0, 1, 1003)
    ws, behind = guard[:need], guard[need:]
    s3r.s3r_workspace_init(ws)
    case.ws = ws
    for pad in (0, 60, 1000):
        ids = torch.tensor([-1, 4] * (pad // 2) + [2, 0, 3, 1], dtype=torch.int32, device="cuda")
        batch = s3r.make_batch(case.seq_lens, case.page_table, req_ids=ids)
        res = run_draft(case, 8, [2, 0, 1, 3], idx, n, seed=5, batch=batch)
        assert s3r.s3r_get_error(ws) == (1 << 5 if pad else 0)
        check_draft(case, 8, [2, 0, 1, 3], idx, n, *res)
        assert (behind == 0x5A).all()


def test_append_and_verify_over_more_entries_than_a_launch_takes():
    """Four requests behind hundreds of empty entries, across the 256 of one verify launch."""
    case = KV8Case(2, 128, [500, 40, 900, 10], 3, seed=16).cuda(8)
    kn, vn = rows(case, 3, seed=5)
    for pad in (254, 700):
        ids = torch.tensor([s3r.NO_REQUEST] * pad + [2, 0, 3, 1], dtype=torch.int32, device="cuda")
        batch = s3r.make_batch(case.seq_lens, case.page_table, req_ids=ids)
        before = state(case)
        s3r.s3r_kv8_append(case.cache, batch, kn, vn, case.ws)
        assert_state(case, expect(case, before, case.lens, [3] * 4, kn, vn, range(4)))
        q = torch.randn((4, 3, 8, 128), device="cuda").bfloat16()
        out, lse = torch.empty_like(q), torch.empty((4, 3, 8), device="cuda")
        s3r.s3r_verify_attn_kv8(case.cache, batch, 2, q, out, lse, None, case.ws)
        assert s3r.s3r_get_error(case.ws) == 0
        check_verify(case, 8, 2, q, out, lse, None)


def test_allocation_of_no_tokens():
    """T = 0: every request gets what its committed length lacks, and an empty slot map is one."""
    lens, table = torch.tensor([33, 0, 16], dtype=torch.int32, device="cuda"), torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    pool = s3r.PagePool(9, table)
    pool.grow(s3r.make_batch(lens, table), 0, slot_map=torch.empty((3, 0), dtype=torch.int64, device="cuda"))
    assert pool.check_errors() == 0 and pool.granted.tolist() == [1, 1, 1] and pool.held.tolist() == [3, 0, 1]
    assert table[0, :3].tolist() + table[2, :1].tolist() == [0, 1, 2, 3] and int(pool.free_count) == 5
