"""GPU: bindings refuse rows that several requests share before anything is launched."""
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import KV8Case
from tests.test_gpu_kv8_append import assert_state, rows, state

pytestmark = pytest.mark.gpu


def test_shared_rows_are_refused():
    case = KV8Case(2, 64, [10, 20, 3], 8, seed=9, upto=0).cuda(4, sel_stride=8)
    kn, vn = rows(case, 4, seed=3)
    q = torch.randn((3, 4, 64), device="cuda").bfloat16()
    step, cnt = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones((3, 2), dtype=torch.int32, device="cuda")
    idx, lse = torch.zeros((3, 2, 8), dtype=torch.int32, device="cuda"), torch.zeros((3, 4), device="cuda")
    before, n0 = state(case), s3r.s3r_launch_count()
    for bad in (lambda: s3r.s3r_kv8_append(case.cache, case.batch, kn[:1].expand_as(kn), vn[:1].expand_as(vn), case.ws),
                lambda: s3r.s3r_kv8_append(case.cache, case.batch, kn, vn[:1].expand_as(vn), case.ws),
                lambda: s3r.s3r_sparse_draft_attn_kv8(case.cache, case.batch, step, q[:1].expand_as(q), idx, cnt, torch.empty_like(q), lse, case.ws)):
        with pytest.raises(ValueError):
            bad()
    assert s3r.s3r_launch_count() == n0
    assert_state(case, before)


def test_shared_rows_of_the_bf16_draft_are_refused():
    pools = [torch.zeros((8, 2, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lens, table = torch.full((3,), 5, dtype=torch.int32, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda").view(3, 1)
    cache, batch = s3r.make_cache(*pools, 4), s3r.make_batch(lens, table)
    ws = s3r.new_workspace(s3r.s3r_workspace_size(cache, 3, 1, 1, 1, 8))
    q, kv = torch.zeros((3, 4, 64), device="cuda").bfloat16(), torch.ones((3, 2, 64), device="cuda").bfloat16()
    step, cnt = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones((3, 2), dtype=torch.int32, device="cuda")
    idx = torch.zeros((3, 2, 8), dtype=torch.int32, device="cuda")
    n0 = s3r.s3r_launch_count()
    for a, b, c in ((q[:1].expand_as(q), kv, kv), (q, kv[:1].expand_as(kv), kv[:1].expand_as(kv))):
        with pytest.raises(ValueError):
            s3r.s3r_sparse_draft_attn(cache, batch, step, a, b, c, idx, cnt, torch.empty_like(q), None, ws)
    assert s3r.s3r_launch_count() == n0 and not pools[0].any()
