"""GPU: the 8-bit verify's row sums where page scales of V lie far apart."""
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import KV8Case
from tests.test_gpu_kv8_attention import check_verify, draft_sets, run_draft, run_verify

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


@pytest.mark.parametrize("d", [64, 128])
def test_smallest_v_scales_give_small_outputs_not_zeros(d):
    """V scales of 2^-122 (append writes down to 2^-126): outputs of about 2^-117 are normal bf16 numbers. Each
    is that of the same codes at scales of 2^-2 times 2^-120, but for the roundings of both: 2^-9 of it
    (bf16, twice), and of each weight 2^-11 (a half) and, for the logarithm of the scale (magnitude below
    256: 2^-17 absolute) in its exponent, 2^-17."""
    case = KV8Case(2, d, [700, 40, 5], 8, seed=31).cuda(8, sel_stride=710)
    idx, n = draft_sets(case, [650, 40, 5], seed=3)
    out = []
    for e in (-2, -122):
        case.v_scale.fill_(2.0 ** e)
        q, o, lse = run_draft(case, 8, [1, 0, 2], idx, n, seed=5)
        q2, o2, lse2, _ = run_verify(case, 8, 1, seed=6, scores=False)
        assert s3r.s3r_get_error(case.ws) == 0
        out.append([t.double() * 2.0 ** (-2 - e) for t in (o, o2)] + [lse, lse2])
    top = 448 * 2.0 ** -2
    for a, b in zip(out[0][:2], out[1][:2]):
        assert (a != 0).any() and ((a - b).abs() <= 2.0 ** -8 * a.abs() + (2.0 ** -10 + 2.0 ** -16) * top).all()
        assert ((b.abs() > 0) == (a.abs() > 0)).float().mean() > 0.99
    assert torch.equal(out[0][2], out[1][2])   # the draft's sums do not see V's scales
    # the verify's terms 2^(x - m) carry them in m (below 256: 2^-17 in each exponent)
    assert ((out[0][3] - out[1][3]).abs() <= 2.0 ** -17 + 2.0 ** -21 * (1 + out[0][3].abs())).all()
