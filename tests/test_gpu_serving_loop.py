"""GPU: a serving loop over a short page pool: prompts wait, requests end, slots are used again, rounds are
replayed from one capture; every committed row of every request stays what it was."""
import numpy as np
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import f64
from tests.test_gpu_kv8_round import tensors
from tests.test_gpu_pool_short import D, HKV, HQ, K, VOCAB, Server, first

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv8", [True, False])
def test_serving_loop(kv8):
    slots, total = 4, 15
    s = Server(kv8, total, slots=slots)
    e, pool, rng = s.e, s.pool, np.random.default_rng(3)
    record = [None] * slots            # committed K, V rows of each request, as given
    refused = waited = ended = replays = 0
    still, graph = [t.clone() for t in tensors(slots, K, HQ, HKV, D, VOCAB, seed=0)], None
    for it in range(60):
        new = False
        for r in range(slots):
            if record[r] is None and rng.random() < 0.5:
                n = int(rng.integers(1, 60))
                pool.grow(s.ids(r), n)
                if int(pool.granted[r]) == 0:
                    waited += 1
                    continue
                rows = [torch.randn((slots, n, HKV, D), device="cuda").bfloat16() for _ in range(2)]
                if kv8:
                    s3r.s3r_kv8_append(e.cache8, s.ids(r), *rows, e.ws)
                else:
                    at = torch.arange(n, device="cuda")
                    for p, x in zip(s.pools, rows):
                        p[s.table[r, at // 16].long(), :, at % 16] = x[r]
                record[r] = [f64(x[r]) for x in rows]
                s.lens[r] = n
                new = True
        e.set_active([x is not None for x in record])
        data = tensors(slots, K, HQ, HKV, D, VOCAB, seed=1000 + it)
        if new or it == 0:
            e.prefill(*first(data))
        lens0 = s.lens.tolist()
        for a, b in zip(still, data):
            a.copy_(b)
        if graph is None and it == 2:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                e.round(*still)
        if graph is None:
            e.round(*still)
        else:
            graph.replay()
            replays += 1
        assert e.check_errors() == 0 and pool.check_errors() == 0
        granted, n_out, lens, held = (t.tolist() for t in (pool.granted, e.buf.n_out, s.lens, pool.held))
        for r in range(slots):
            if not granted[r] or record[r] is None:
                assert n_out[r] == 0 and lens[r] == lens0[r]
                refused += record[r] is not None
            else:
                assert n_out[r] > 0 and lens[r] == lens0[r] + n_out[r] and held[r] >= -(-lens[r] // 16)
                s.check_verify(r, lens0[r], data[0])
                record[r] = [np.concatenate([a, f64(b[r, :n_out[r]])]) for a, b in zip(record[r], data[1:3])]
            if record[r] is None:
                continue
            for got, want in zip(s.rows(r, lens[r]), record[r]):
                want = want.transpose(1, 0, 2)
                if not kv8:
                    np.testing.assert_array_equal(got, want)
                else:   # e4m3's half step, and half of its smallest step for each of a page's rewritings
                    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 8 * K * 2.0 ** -17).all()
            if lens[r] + K + 2 > 7 * 16 or rng.random() < 0.08 or (not granted[r] and rng.random() < 0.3):
                keep = [x is not None and q != r for q, x in enumerate(record)]
                e.set_active(keep)
                pool.release(s.ids(r))
                s.lens[r], record[r] = 0, None
                ended += 1
        used = sum((s.table[r, :h].tolist() for r, h in enumerate(pool.held.tolist())), [])
        assert sorted(used + pool.free_pages[:int(pool.free_count)].tolist()) == list(range(total))
    assert refused > 3 and waited > 0 and ended > 3 and replays > 50
