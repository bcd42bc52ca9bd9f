"""GPU: every draft step of an engine's rounds over an 8-bit cache, against 64-bit attention over the cache
as it stands at that step and with the attention tests' own bounds; every set against the oracle's."""
import numpy as np
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from oracle import s3r_oracle as O
from tests.kv8_testlib import DRAFT, KV8Case, assert_within, attention_bounds, f64
from tests.test_gpu_kv8_round import engine, tensors

pytestmark = pytest.mark.gpu


def position_scores(e, lens, k):
    """sigma of every committed position from the engine's last logits (lengths `lens`)."""
    b = e.buf
    batch = s3r.make_batch(lens, e.page_table)
    NR, Hq, Hkv, _, cap = b.dims
    logits = b._scores[: NR * Hq * (k + 1) * cap].view(NR, Hkv, -1, cap)
    lse = b.prefill_lse if k == 0 else b.lse
    out = torch.zeros((NR, Hkv, cap), device="cuda")
    s3r.s3r_position_scores(e.cache, batch, logits, lse, k, out, e.ws)
    return out.cpu().numpy()


@pytest.mark.parametrize("Hq,Hkv,d,k,lens,kw", [
    (8, 2, 128, 6, [500, 1300, 90], {}),
    (4, 1, 64, 3, [200, 257], dict(page_select=True)),
    (16, 2, 128, 2, [40, 700, 33], dict(greedy=True, overlap_scores=False)),
    (64, 8, 64, 4, [31, 16, 170], dict(page_select=True, overlap_scores=False)),
])
def test_every_draft_step_reads_its_own_row_and_the_set(Hq, Hkv, d, k, lens, kw):
    case = KV8Case(Hkv, d, lens, 60, seed=sum(lens), upto=0).cuda(Hq)
    e = engine(case, Hq, k, **kw)
    nr, G, b = case.nr, Hq // Hkv, e.buf
    q, kb, vb, p, ql = tensors(nr, k, Hq, Hkv, d, 512, seed=3)
    e.prefill(q[:, :1].contiguous(), kb[:, :1].contiguous(), vb[:, :1].contiguous())
    prev, seen = case.seq_lens.clone(), 0
    for it in range(3):
        q, kb, vb, p, ql = tensors(nr, k, Hq, Hkv, d, 512, seed=50 + it)
        L0 = case.seq_lens.tolist()
        sigma = position_scores(e, prev, e.k_prev)
        e.select()
        sets = [[b.sel_idx[r, h, : int(b.sel_count[r, h])].cpu().numpy().astype(int) for h in range(Hkv)] for r in range(nr)]
        choose = O.select_pages if kw.get("page_select") else O.select_positions
        for r in range(nr):
            for h in range(Hkv):
                np.testing.assert_array_equal(sets[r][h], choose(sigma[r, h], L0[r], 1000, 32))
        for i in range(k):
            e.draft_step(i, q, kb, vb, ql)
            got, got_lse = f64(b.draft_out), f64(b.draft_lse)
            for r in range(nr):
                K, V = case.values(r, L0[r] + i + 1)
                for h in range(Hkv):
                    at = np.concatenate([sets[r][h], np.arange(L0[r], L0[r] + i + 1)])
                    rows = f64(q[r, i])[h * G:(h + 1) * G][None]
                    o, l, _, bo, bl, _ = attention_bounds(rows, K[h:h + 1, at], V[h:h + 1, at], np.ones((G, at.size), bool), **DRAFT)
                    assert_within(got[r, h * G:(h + 1) * G][None], o, bo, f"draft it={it} i={i} r={r} h={h}")
                    assert_within(got_lse[r, h * G:(h + 1) * G][None], l, bl, f"lse it={it} i={i} r={r} h={h}")
                    # without the step's own row the result would lie outside
                    o1 = attention_bounds(rows, K[h:h + 1, at[:-1]], V[h:h + 1, at[:-1]], np.ones((G, at.size - 1), bool), **DRAFT)[0]
                    assert (np.abs(o1 - o) > 2 * bo).any()
                    seen += 1
        prev = case.seq_lens.clone()
        e.verify(q, kb, vb)
        e.sample_and_commit(p, ql)
        assert e.check_errors() == 0
    assert seen == 3 * k * nr * Hkv
