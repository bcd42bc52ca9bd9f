"""GPU: a prefill between rounds (a batch slot that goes to a new request)."""
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import KV8Case
from tests.test_gpu_kv8_round import engine, tensors

pytestmark = pytest.mark.gpu


# (a round captured without overlapped scores selects from a verify's: captured again after a prefill)
@pytest.mark.parametrize("captured,kw", [(False, {}), (False, dict(page_select=True)), (False, dict(overlap_scores=False)),
                                         (True, {}), (True, dict(page_select=True))])
def test_the_round_after_another_prefill_selects_from_its_scores(captured, kw):
    """Two engines over equal caches do rounds, and then one of them is given another query for a
    prefill: the next round's sets are those of an engine whose first prefill it is."""
    k, dims = 3, (8, 2, 128)
    data = [tensors(3, k, *dims, 512, seed=40 + i) for i in range(3)]

    def first(x):
        return [t[:, :1].contiguous() for t in x[:3]]

    case = KV8Case(2, 128, [500, 700, 90], 60, seed=3, upto=0).cuda(8)
    e = engine(case, 8, k, **kw)
    e.prefill(*first(data[0]))
    e.round(*data[0])
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            e.round(*data[2])
    e.prefill(*first(data[1]))
    # a fresh engine on a copy of the caches as they are now
    twin = KV8Case(2, 128, [500, 700, 90], 60, seed=3, upto=0)
    twin.cuda(8)
    for name in ("k", "v", "k_scale", "v_scale", "seq_lens"):
        getattr(twin, name).copy_(getattr(case, name))
    f = engine(twin, 8, k, **kw)
    f.prefill(*first(data[1]))
    if captured:
        graph.replay()
    else:
        e.round(*data[2])
    f.round(*data[2])
    assert e.check_errors() == 0 and f.check_errors() == 0
    assert torch.equal(e.buf.sel_count, f.buf.sel_count)
    for r in range(3):
        for h in range(2):
            n = int(e.buf.sel_count[r, h])
            assert torch.equal(e.buf.sel_idx[r, h, :n], f.buf.sel_idx[r, h, :n])
    assert torch.equal(e.buf.draft_out, f.buf.draft_out) and torch.equal(e.buf.verify_out, f.buf.verify_out)
    assert torch.equal(e.seq_lens, f.seq_lens)
