"""GPU: the 8-bit verify's row sums where page scales of V lie far apart."""
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import KV8Case
from tests.test_gpu_kv8_attention import check_verify, run_verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("period,low", [(8, 4), (16, 12), (12, 9)])
def test_far_v_scales_leave_the_normaliser_alone(period, low):
    """Of every `period` tiles the first `low` hold V scales of 2^-119 and the others of 2^40: a span's
    first chunk far below its second, spans far below others. The low pages count as zeros in the
    output (2^-159 of the others), their weights count in the sums like any other."""
    case = KV8Case(8, 128, [9000, 12000, 7000, 10000, 30000], 7, seed=29).cuda(32)
    for r in range(case.nr):
        at = [[int(x) for i, x in enumerate(case.pt[r]) if x >= 0 and (i // 8 % period < low) == side] for side in (True, False)]
        case.v_scale[torch.tensor(at[0], device="cuda")] = 2.0 ** -119
        case.v_scale[torch.tensor(at[1], device="cuda")] = 2.0 ** 40
    res = run_verify(case, 32, 6, seed=13, scores=False)
    assert s3r.s3r_get_error(case.ws) == 0
    check_verify(case, 32, 6, *res)
