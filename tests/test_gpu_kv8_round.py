"""GPU: whole rounds over the 8-bit cache and over page tables that grow on the GPU."""
import numpy as np
import pytest
import torch

import synth
import sparse_dense_kv_b200 as s3r
from oracle import s3r_oracle as O
from tests.kv8_testlib import DRAFT, K8, VERIFY, KV8Case, assert_within, attention_bounds, f64, rows_of

pytestmark = pytest.mark.gpu


def tensors(nr, k, Hq, Hkv, d, vocab, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, kb, vb = r(nr, k + 1, Hq, d).bfloat16(), r(nr, k + 1, Hkv, d).bfloat16(), r(nr, k + 1, Hkv, d).bfloat16()
    p = r(nr, k + 1, vocab) * 1.5
    return q, kb, vb, p, (p[:, :k] + 0.4 * r(nr, k, vocab)).contiguous()


def engine(case, Hq, k, **kw):
    d = dict(k=k, budget_bp=1000, window=32, vocab=512, seed=77)
    d.update(kw)
    return s3r.S3REngine(case.k, case.v, case.page_table, case.seq_lens, Hq, k_scale=case.k_scale, v_scale=case.v_scale, **d)


@pytest.mark.parametrize("Hq,Hkv,d,k,lens,kw", [
    (8, 2, 128, 6, [500, 1300, 90], {}),
    (4, 1, 64, 3, [200, 257], dict(page_select=True)),
    (16, 2, 128, 2, [40, 700], dict(greedy=True, overlap_scores=False)),
])
def test_rounds_match_64_bit_attention_and_the_bf16_cache_s_decisions(Hq, Hkv, d, k, lens, kw):
    """Rounds of an engine on an 8-bit cache: each verify and the last draft step against 64-bit
    attention over the cache's values, the sets against the oracle's selection from the same
    scores, and the tokens against an engine on a bf16 cache given the same logits (sampling
    sees nothing of the cache)."""
    case = KV8Case(Hkv, d, lens, 60, seed=sum(lens), upto=0).cuda(Hq)
    e = engine(case, Hq, k, **kw)
    nr, G = case.nr, Hq // Hkv
    total, mp = case.total, case.max_pages
    bf = s3r.S3REngine(torch.randn((total, Hkv, 16, d), device="cuda").bfloat16(), torch.randn((total, Hkv, 16, d), device="cuda").bfloat16(),
                       case.page_table, case.seq_lens.clone(), Hq, k=k, budget_bp=1000, window=32, vocab=512, seed=77, **kw)
    q, kb, vb, p, ql = tensors(nr, k, Hq, Hkv, d, 512, seed=3)
    for eng in (e, bf):
        eng.prefill(q[:, :1].contiguous(), kb[:, :1].contiguous(), vb[:, :1].contiguous())
    for it in range(3):
        q, kb, vb, p, ql = tensors(nr, k, Hq, Hkv, d, 512, seed=10 + it)
        lens0 = case.seq_lens.cpu().numpy().astype(int)
        ready, pos = e._scores_ready, e.pos_scores.clone() if e.overlap_scores else None
        n0 = s3r.s3r_launch_count()
        e.round(q, kb, vb, p, ql)
        n1 = s3r.s3r_launch_count()
        assert n1 - n0 == e.launches_per_round + (1 if e.overlap_scores and not ready else 0)
        bf.round(q, kb, vb, p, ql)
        assert e.check_errors() == 0
        assert torch.equal(e.buf.draft_tokens, bf.buf.draft_tokens) and torch.equal(e.buf.n_out, bf.buf.n_out)
        for r in range(nr):
            n = int(e.buf.n_out[r])
            assert torch.equal(e.buf.out_tokens[r, :n], bf.buf.out_tokens[r, :n])
            L, T = lens0[r], k + 1
            K, V = case.values(r, L + T)
            vis = np.arange(L + T)[None, :] <= L + (np.arange(G * T) // G)[:, None]
            o, l, x, bo, bl, bx = attention_bounds(rows_of(f64(q[r]), Hkv), K, V, vis, **VERIFY)
            assert_within(rows_of(f64(e.buf.verify_out[r]), Hkv), o, bo, f"verify r={r} it={it}")
            assert_within(f64(e.buf.scores[r])[:, :, :L], x[:, :, :L], bx[:, :, :L] + 1e-30, "scores")
            for h in range(Hkv):
                cnt = int(e.buf.sel_count[r, h])
                sel = e.buf.sel_idx[r, h, :cnt].cpu().numpy().astype(int)
                if pos is not None and ready and not kw.get("page_select"):
                    want = O.select_positions(pos[r, h].cpu().numpy()[:L], L, 1000, 32)
                    np.testing.assert_array_equal(sel, want)
                at = np.concatenate([sel, np.arange(L, L + k)])
                # (the verify rewrote the block's rows from the same bf16 rows, beside one more: a page's
                # scale may have moved, which moves codes under the normal range by half a step at most)
                rows = f64(q[r, k - 1])[h * G:(h + 1) * G][None]
                o, l, _, bo, bl, _ = attention_bounds(rows, K[h:h + 1, at], V[h:h + 1, at], np.ones((G, at.size), bool), **DRAFT)
                slack = 2.0 ** -4 * np.abs(V[h, at[-k - 16:]]).max() * (k + 16) / at.size + 0.05
                assert np.abs(f64(e.buf.draft_out[r])[h * G:(h + 1) * G] - o[0]).max() <= bo.max() + slack


def test_captured_rounds_replay_what_eager_rounds_do():
    """One captured round replayed from the start state gives bit for bit what eager rounds give;
    two engines' graphs (own workspaces) interleaved on two streams do not disturb each other."""
    outs = []
    for mode in ("eager", "graph", "two"):
        cases = [KV8Case(2, 128, [400, 900], 60, seed=5 + j, upto=0).cuda(8) for j in range(2)]
        engs = [engine(c, 8, 4) for c in cases]
        data = [tensors(2, 4, 8, 2, 128, 512, seed=20 + j) for j in range(2)]
        for e, (q, kb, vb, p, ql) in zip(engs, data):
            e.prefill(q[:, :1].contiguous(), kb[:, :1].contiguous(), vb[:, :1].contiguous())
            e.round(q, kb, vb, p, ql)
        torch.cuda.synchronize()
        if mode == "eager":
            for _ in range(3):
                for e, x in zip(engs, data):
                    e.round(*x)
        else:
            graphs = []
            for e, x in zip(engs, data):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    e.round(*x)
                graphs.append(g)
            streams = [torch.cuda.Stream() for _ in engs] if mode == "two" else [torch.cuda.current_stream()] * 2
            for s in streams:
                s.wait_stream(torch.cuda.current_stream())
            for _ in range(3):
                for g, s in zip(graphs, streams):
                    with torch.cuda.stream(s):
                        g.replay()
        torch.cuda.synchronize()
        assert all(e.check_errors() == 0 for e in engs)
        outs.append([t.clone() for e, c in zip(engs, cases) for t in (e.buf.verify_out, e.buf.lse, e.buf.draft_out, e.seq_lens, e.buf.n_out,
                                                                      c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)])
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


def test_mixed_phases_and_another_stream():
    """Subsets of an 8-bit batch at different phases, on a side stream: every request's verify
    output is that of 64-bit attention."""
    case = KV8Case(2, 64, [300, 77, 512, 130], 60, seed=9, upto=0).cuda(4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        e = engine(case, 4, 2)
        q, kb, vb, p, ql = tensors(4, 2, 4, 2, 64, 512, seed=1)
        e.prefill(q[:, :1].contiguous(), kb[:, :1].contiguous(), vb[:, :1].contiguous())
        drv = s3r.MixedPhaseDriver(e, [0, 1, 2, 1])
        drv.start(q, kb, vb, ql)
        for _ in range(6):
            lens0 = case.seq_lens.cpu().numpy().astype(int)
            done = drv.iterate(q, kb, vb, p, ql)
            for r in done:
                K, V = case.values(r, lens0[r] + 3)
                vis = np.arange(lens0[r] + 3)[None, :] <= lens0[r] + (np.arange(6) // 2)[:, None]
                o, l, x, bo, bl, bx = attention_bounds(rows_of(f64(q[r]), 2), K, V, vis, **VERIFY)
                assert_within(rows_of(f64(e.buf.verify_out[r]), 2), o, bo, f"r={r}")
        assert e.check_errors() == 0


@pytest.mark.parametrize("kv8", [True, False])
def test_rounds_over_tables_that_grow_on_the_gpu(kv8):
    """Captured rounds over a page pool: the tables follow the lengths across page edges, the outputs
    are those of an engine whose pages were all there, and everything comes back at the end."""
    Hq, Hkv, d, k, lens, total = 8, 2, 128, 3, [0, 15, 30], 40
    outs = []
    for grown in (True, False):
        pools = [torch.zeros((total, Hkv, 16, d), dtype=torch.uint8 if kv8 else torch.bfloat16, device="cuda") for _ in range(2)]
        sc = [torch.ones((total, Hkv), device="cuda") for _ in range(2)]
        table = torch.full((3, 12), -1, dtype=torch.int32, device="cuda")
        seq = torch.zeros(3, dtype=torch.int32, device="cuda")
        batch = s3r.make_batch(seq, table)
        pool = s3r.PagePool(total, table) if grown else None
        if grown:
            pool.grow(batch, max(lens), n_new=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        else:
            table.copy_(torch.arange(36, dtype=torch.int32).view(3, 12))
        kw = dict(k_scale=sc[0], v_scale=sc[1]) if kv8 else {}
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        e = s3r.S3REngine(*pools, table, seq, Hq, k=k, budget_bp=5000, window=8, vocab=512, seed=5, pages=pool, **kw)
        q, kb, vb, p, ql = tensors(3, k, Hq, Hkv, d, 512, seed=4)
        # the prompts' rows: zeros are in the pools already (scale 1)
        e.prefill(q[:, :1].contiguous(), kb[:, :1].contiguous(), vb[:, :1].contiguous())
        e.round(q, kb, vb, p, ql)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            e.round(q, kb, vb, p, ql)
        for _ in range(8):
            g.replay()
        assert e.check_errors() == 0
        outs.append([t.clone() for t in (e.buf.verify_out, e.buf.lse, e.buf.sel_idx, e.seq_lens, e.buf.n_out)])
        if grown:
            assert pool.check_errors() == 0 and (pool.granted == 1).all()
            held, L = pool.held.cpu().numpy(), seq.cpu().numpy()
            assert (held >= -(-L // 16)).all() and (held <= -(-(L + k + 1) // 16)).all()
            assert int(pool.free_count) == total - held.sum()
            used = [table[r, :held[r]].tolist() for r in range(3)]
            assert len(set(sum(used, []))) == held.sum()
            pool.release(batch)
            assert int(pool.free_count) == total and sorted(pool.free_pages.tolist()) == list(range(total))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_engine_refuses_half_an_8_bit_cache():
    case = KV8Case(1, 64, [20], 4, seed=1).cuda(1)
    with pytest.raises(ValueError):
        s3r.S3REngine(case.k, case.v, case.page_table, case.seq_lens, 1, k=1, budget_bp=100, window=4, vocab=64, seed=1, k_scale=case.k_scale)
    with pytest.raises(ValueError):
        engine(case, 1, 1, pages=s3r.PagePool(4, case.page_table.clone()))
