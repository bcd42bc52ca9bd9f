"""GPU: rounds over a page pool that runs short: slots used again, refused requests, idle slots."""
import numpy as np
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import K8, VERIFY, assert_within, attention_bounds, f64, rows_of
from tests.test_gpu_kv8_round import tensors

pytestmark = pytest.mark.gpu

HQ, HKV, D, K, VOCAB, COLS = 8, 2, 128, 3, 512, 8


class Server:
    """A batch of slots over one pool; prompts are random rows, the same for a slot and length."""

    def __init__(self, kv8, total, slots=3, **kw):
        self.kv8 = kv8
        g = torch.Generator(device="cuda").manual_seed(1)
        if kv8:
            self.pools = [torch.randint(0, 120, (total, HKV, 16, D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
            self.scales = [torch.full((total, HKV), 2.0 ** -7, device="cuda") for _ in range(2)]
        else:
            self.pools = [torch.randn((total, HKV, 16, D), generator=g, device="cuda").bfloat16() for _ in range(2)]
            self.scales = []
        self.table = torch.full((slots, COLS), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(slots, dtype=torch.int32, device="cuda")
        self.batch = s3r.make_batch(self.lens, self.table)
        self.pool = s3r.PagePool(total, self.table)
        skw = dict(k_scale=self.scales[0], v_scale=self.scales[1]) if kv8 else {}
        self.e = s3r.S3REngine(*self.pools, self.table, self.lens, HQ, k=K, budget_bp=5000, window=8, vocab=VOCAB, seed=5, pages=self.pool,
                               **skw, **kw)

    def ids(self, *slots):
        return s3r.make_batch(self.lens, self.table, req_ids=torch.tensor(slots, dtype=torch.int32, device="cuda"))

    def admit(self, slot, n):
        """Pages and prompt rows for n more tokens of a slot."""
        L = int(self.lens[slot])
        self.pool.grow(self.ids(slot), n)
        assert int(self.pool.granted[slot]) == 1
        g = torch.Generator(device="cuda").manual_seed(100 * slot + n)
        rows = [torch.randn((3, n, HKV, D), generator=g, device="cuda").bfloat16() for _ in range(2)]
        if self.kv8:
            s3r.s3r_kv8_append(self.e.cache8, self.ids(slot), *rows, self.e.ws)
        else:
            for pool, x in zip(self.pools, rows):
                for t in range(n):
                    pool[int(self.table[slot, (L + t) // 16]), :, (L + t) % 16] = x[slot, t]
        self.lens[slot] += n

    def rows(self, slot, n):
        """K, V [HKV][n][D] in 64 bits."""
        pages = self.table[slot].cpu().numpy()
        if self.kv8:
            return [K8.dequantise(p.cpu().numpy(), s.cpu().numpy(), pages, n) for p, s in zip(self.pools, self.scales)]
        return [f64(p)[pages[:-(-n // 16)]].transpose(1, 0, 2, 3).reshape(HKV, -1, D)[:, :n] for p in self.pools]

    def check_verify(self, slot, L, q):
        G, T = HQ // HKV, K + 1
        kk, vv = self.rows(slot, L + T)
        vis = np.arange(L + T)[None, :] <= L + (np.arange(G * T) // G)[:, None]
        o, lse, _, bo, bl, _ = attention_bounds(rows_of(f64(q[slot]), HKV), kk, vv, vis, **VERIFY)
        assert_within(rows_of(f64(self.e.buf.verify_out[slot]), HKV), o, bo, f"slot {slot}")

    def everything(self):
        return [t.clone() for t in (*self.pools, *self.scales)]


def first(x):
    return [t[:, :1].contiguous() for t in x[:3]]


def crowded(kv8, with_third, **kw):
    """Seven pages: slot 2 held three, gave them back, and they went to slots 0 and 1; then slot 2 got
    one page again. Its table row still names the other two behind it. With `with_third` false slot
    2 holds a page and is no part of the engine's rounds."""
    s = Server(kv8, 7, **kw)
    s.admit(0, 10)
    s.admit(1, 33)
    s.admit(2, 40)
    s.pool.release(s.ids(2))
    s.lens[2] = 0
    s.admit(1, 17)
    s.admit(0, 10)
    s.admit(2, 16)
    assert s.pool.held.tolist() == [2, 4, 1] and int(s.pool.free_count) == 0
    stale, others = set(s.table[2, 1:3].tolist()), set(s.table[0, :2].tolist() + s.table[1, :4].tolist())
    assert stale <= others
    if not with_third:
        s.e.set_active([1, 1, 0])
    return s


@pytest.mark.parametrize("kw", [dict(), dict(greedy=True), dict(overlap_scores=False, page_select=True)])
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kv8", [True, False])
def test_a_refused_request_touches_nothing_and_goes_on_later(kv8, captured, kw):
    data = [tensors(3, K, HQ, HKV, D, VOCAB, seed=60 + i) for i in range(6)]
    still = [t.clone() for t in data[0]]
    runs = []
    for third in (True, False):
        s = crowded(kv8, third, **kw)
        e = s.e
        e.prefill(*first(data[0]))
        e.round(*data[1])
        graph = None
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                e.round(*still)
        trail = []
        for x in data[2:4]:
            if captured:
                for a, b in zip(still, x):
                    a.copy_(b)
                graph.replay()
            else:
                e.round(*x)
            assert e.check_errors() == 0 and s.pool.check_errors() == 0
            trail.append([t[:2].clone() for t in (e.buf.verify_out, e.buf.lse, e.buf.out_tokens, e.buf.n_out, s.lens, e.buf.draft_out)])
            assert int(s.lens[2]) == 16 and int(e.buf.n_out[2]) == 0 and (e.buf.n_out[:2] > 0).all()
        assert s.pool.granted.tolist() == [1, 1, 0] and s.pool.held.tolist()[2] == 1
        runs.append((s.everything(), trail, s, e, graph))
    for a, b in zip(runs[0][0], runs[1][0]):   # every page of the pool
        assert torch.equal(a, b)
    for a, b in zip(runs[0][1], runs[1][1]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))

    # slot 0 ends: its pages stay with the pool until slot 2 needs them
    s, e, graph = runs[0][2:]
    e.set_active([0, 1, 1])
    s.pool.release(s.ids(0))
    if kw.get("overlap_scores") is not False or not captured:
        e.prefill(*first(data[4]))
    for x in data[4:6]:
        L = s.lens.tolist()
        if captured:
            for a, b in zip(still, x):
                a.copy_(b)
            graph.replay()
        else:
            e.round(*x)
        assert e.check_errors() == 0 and s.pool.check_errors() == 0
        assert s.pool.granted.tolist() == [0, 1, 1] and int(s.pool.held[0]) == 0 and int(s.lens[0]) == L[0]
        assert e.buf.n_out[0] == 0 and (s.lens[1:].cpu() - torch.tensor(L[1:]) == e.buf.n_out[1:].cpu()).all() and (e.buf.n_out[1:] > 0).all()
        for slot in (1, 2):
            s.check_verify(slot, L[slot], x[0])
    held = s.pool.held.tolist()
    used = [s.table[r, :held[r]].tolist() for r in range(3)]
    assert len(set(sum(used, []))) == sum(held) and int(s.pool.free_count) == 7 - sum(held)


@pytest.mark.parametrize("kv8", [True, False])
def test_a_request_refused_at_its_prefill_waits(kv8):
    """No page for a slot's pending token: its prefill writes nothing; the slot's first rounds, once there
    are pages, are right without another prefill."""
    data = [tensors(3, K, HQ, HKV, D, VOCAB, seed=80 + i) for i in range(4)]
    s = crowded(kv8, True)
    before = s.everything()
    kept = sorted(set(range(7)) - set(s.table[0, :2].tolist() + s.table[1, :4].tolist()))
    s.e.prefill(*first(data[0]))
    assert s.e.check_errors() == 0 and s.pool.check_errors() == 0 and s.pool.granted.tolist() == [1, 1, 0]
    for a, b in zip(before, s.everything()):
        assert torch.equal(a[kept], b[kept])
    s.e.round(*data[1])
    s.e.set_active([0, 1, 1])
    s.pool.release(s.ids(0))
    for x in data[2:]:
        L = s.lens.tolist()
        s.e.round(*x)
        assert s.e.check_errors() == 0 and int(s.e.buf.n_out[2]) > 0
        for slot in (1, 2):
            s.check_verify(slot, L[slot], x[0])


def test_idle_slots_take_no_pages_and_wake_up():
    s = Server(True, 20)
    s.admit(1, 30)
    s.e.set_active([0, 1, 0])
    data = [tensors(3, K, HQ, HKV, D, VOCAB, seed=90 + i) for i in range(4)]
    s.e.prefill(*first(data[0]))
    s.e.round(*data[1])
    assert s.pool.held.tolist() == [0, 3, 0] and s.pool.granted.tolist() == [0, 1, 0] and s.lens.tolist()[::2] == [0, 0]
    s.admit(0, 20)
    s.e.set_active(torch.tensor([True, True, False]))
    s.e.prefill(*first(data[2]))
    L = s.lens.tolist()
    s.e.round(*data[3])
    for slot in (0, 1):
        s.check_verify(slot, L[slot], data[3][0])
    assert s.e.check_errors() == 0 and int(s.pool.held[2]) == 0 and int(s.lens[2]) == 0


def test_pool_and_engine_refusals():
    s = Server(True, 8)
    with pytest.raises(ValueError):
        s.e.set_active([1, 1])
    with pytest.raises(ValueError):
        s.pool.grow(s3r.make_batch(s.lens, s.table.clone()), 1)       # another table
    with pytest.raises(ValueError):
        s.pool.release(s3r.make_batch(s.lens, s.table.clone()))
    big = s3r.PagePool(9, s.table)                                    # more pages than the cache has
    args = (*s.pools, s.table, s.lens, HQ)
    kw = dict(k=K, budget_bp=5000, window=8, vocab=VOCAB, seed=5, k_scale=s.scales[0], v_scale=s.scales[1])
    with pytest.raises(ValueError):
        s3r.S3REngine(*args, pages=big, **kw)
    with pytest.raises(ValueError):
        s3r.S3REngine(*args, **kw).set_active([1, 1, 1])              # no pool


def test_prompts_of_a_whole_batch_are_admitted_as_far_as_the_pool_goes():
    """One allocation and one append for all prompts over the served list, then rounds recorded by
    S3REngine.capture; the prompt that found no pages is admitted when another one has ended."""
    nr, total = 3, 6
    pools = [torch.full((total, HKV, 16, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]     # NaN codes: nothing was written
    scales = [torch.ones((total, HKV), device="cuda") for _ in range(2)]
    table, lens = torch.full((nr, COLS), -1, dtype=torch.int32, device="cuda"), torch.zeros(nr, dtype=torch.int32, device="cuda")
    pool, batch = s3r.PagePool(total, table), s3r.make_batch(lens, table)
    n = torch.tensor([20, 70, 17], dtype=torch.int32, device="cuda")        # 2, 5 and 2 pages
    pool.grow(batch, 70, n_new=n)
    assert pool.granted.tolist() == [1, 0, 0] and pool.served().tolist() == [0, s3r.NO_REQUEST, s3r.NO_REQUEST]
    pool.grow(s3r.make_batch(lens, table, req_ids=torch.tensor([2], dtype=torch.int32, device="cuda")), 70, n_new=n)
    e = s3r.S3REngine(*pools, table, lens, HQ, k=K, budget_bp=5000, window=8, vocab=VOCAB, seed=5, k_scale=scales[0], v_scale=scales[1], pages=pool)
    g = torch.Generator(device="cuda").manual_seed(7)
    kp, vp = (torch.randn((nr, 70, HKV, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    assert pool.served().tolist() == [0, s3r.NO_REQUEST, 2]
    s3r.s3r_kv8_append(e.cache8, s3r.make_batch(lens, table, req_ids=pool.served()), kp, vp, pool.ws, n_new=n)
    lens.copy_(n * pool.granted)
    e.set_active(pool.granted)
    data = [tensors(nr, K, HQ, HKV, D, VOCAB, seed=110 + i) for i in range(2)]
    e.prefill(*first(data[0]))
    e.round(*data[1])
    graph, launches = e.capture(lambda: e.round(*data[1]))                  # (runs the round once more)
    assert launches == e.launches_per_round
    graph.replay()
    assert e.check_errors() == 0 and pool.check_errors() == 0
    assert lens.tolist()[1] == 0 and e.buf.n_out[1] == 0 and min(lens.tolist()[::2]) >= 20
    # the first ends
    e.set_active([0, 0, 1])
    pool.release(s3r.make_batch(lens, table, req_ids=torch.tensor([0], dtype=torch.int32, device="cuda")))
    lens[0], n[1] = 0, 30
    one = s3r.make_batch(lens, table, req_ids=torch.tensor([1], dtype=torch.int32, device="cuda"))
    pool.grow(one, 70, n_new=n)
    assert int(pool.granted[1]) == 1
    s3r.s3r_kv8_append(e.cache8, one, kp, vp, e.ws, n_new=n)
    lens[1] = 30
    e.set_active([0, 1, 1])
    e.prefill(*first(data[0]))
    before = lens.tolist()
    graph.replay()
    assert e.check_errors() == 0 and pool.check_errors() == 0 and pool.granted.tolist() == [0, 1, 1]
    assert lens.tolist()[0] == 0 and lens.tolist()[1] > 30 and lens.tolist()[2] > before[2] and int(pool.held[0]) == 0
    assert not e.buf.verify_out[1:].isnan().any()
