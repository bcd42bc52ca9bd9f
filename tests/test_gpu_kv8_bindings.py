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
