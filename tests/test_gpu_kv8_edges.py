"""GPU: calls at the edges of what the 8-bit cache's documentation allows."""
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import KV8Case
from tests.test_gpu_kv8_append import assert_state, expect, rows, state

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
