"""GPU: empty entries (NO_REQUEST) in the request list of every call: skipped without a report, the other
requests' results those of a list without them."""
import numpy as np
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.test_gpu_kv8_round import tensors

pytestmark = pytest.mark.gpu
NONE = s3r.NO_REQUEST


def one_round(kv8, ids, greedy, page_select):
    """Every call of a round over the given list, from the same start; all that it may write."""
    NR, Hq, Hkv, d, k, V = 4, 8, 2, 128, 2, 512
    g = torch.Generator(device="cuda").manual_seed(2)
    lens = torch.tensor([70, 300, 33, 150], dtype=torch.int32, device="cuda")
    table = torch.arange(NR * 24, dtype=torch.int32, device="cuda").view(NR, 24)
    shape = (NR * 24, Hkv, 16, d)
    if kv8:
        pools = [torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        scales = [torch.full(shape[:2], 2.0 ** -7, device="cuda") for _ in range(2)]
    else:
        pools, scales = [torch.randn(shape, generator=g, device="cuda").bfloat16() for _ in range(2)], []
    kw = dict(k_scale=scales[0], v_scale=scales[1]) if kv8 else {}
    e = s3r.S3REngine(*pools, table, lens, Hq, k=k, budget_bp=3000, window=16, vocab=V, seed=3, greedy=greedy, page_select=page_select, **kw)
    for t in (e.buf._scores, e.buf._lse, e.buf._verify_out, e.buf.prefill_lse, e.buf.draft_out, e.buf.draft_lse, e.pos_scores):
        t.zero_()
    t = torch.tensor(ids, dtype=torch.int32, device="cuda")
    e.batch, e._snap_batch = s3r.make_batch(lens, table, req_ids=t), s3r.make_batch(e._len_snap, table, req_ids=t)
    q, kb, vb, p, ql = tensors(NR, k, Hq, Hkv, d, V, seed=4)
    out = e.prefill(q[:, :1].contiguous(), kb[:, :1].contiguous(), vb[:, :1].contiguous())
    out[[r for r in range(NR) if r not in ids]] = 0
    e.round(q, kb, vb, p, ql)      # selects by s3r_select_kv
    e.round(q, kb, vb, p, ql)      # selects from position scores
    b = e.buf
    return e.check_errors(), [out, *pools, *scales, lens, b.scores, b.lse, b.verify_out, b.sel_idx, b.sel_count, b.draft_out, b.draft_lse,
                              b.draft_tokens, b.out_tokens, b.n_out, b.stats, e.pos_scores]


@pytest.mark.parametrize("greedy,page_select", [(False, False), (True, True)])
@pytest.mark.parametrize("kv8", [True, False])
def test_rounds_over_lists_with_empty_entries(kv8, greedy, page_select):
    err, want = one_round(kv8, [2, 0], greedy, page_select)
    assert err == 0
    for ids in ([NONE, 2, NONE, 0], [2, 0, NONE, NONE, NONE, NONE, NONE]):
        err, got = one_round(kv8, ids, greedy, page_select)
        assert err == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert one_round(kv8, [2, 0, -1], greedy, page_select)[0] == 1 << 5      # an id that is none is still reported
    err, got = one_round(kv8, [NONE] * 3, greedy, page_select)
    assert err == 0 and not got[-2].any()                                    # nobody: no counts


def test_page_calls_over_lists_with_empty_entries():
    lens = torch.tensor([40, 5, 100, 16], dtype=torch.int32, device="cuda")
    got = []
    for ids in ([3, 1, 0], [NONE, 3, 1, NONE, NONE, 0]):
        table = torch.full((4, 10), -1, dtype=torch.int32, device="cuda")
        pool = s3r.PagePool(30, table)
        batch = s3r.make_batch(lens, table, req_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))
        slots = torch.full((4, 7), -9, dtype=torch.int64, device="cuda")
        pool.grow(batch, 7, slot_map=slots)
        a = [t.clone() for t in (table, pool.held, pool.granted, pool.free_count, slots)]
        pool.release(batch, keep_len=torch.tensor([17, 0, 0, 1], dtype=torch.int32, device="cuda"))
        assert pool.check_errors() == 0
        got.append(a + [pool.held, pool.free_count, pool.free_pages])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    np.testing.assert_array_equal(got[0][1].cpu().numpy(), [3, 1, 0, 2])
