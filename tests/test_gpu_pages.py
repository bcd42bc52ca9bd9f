"""GPU: page allocation, slot maps and release against the oracle."""
import numpy as np
import pytest
import torch

import sparse_dense_kv_b200 as s3r
from tests.kv8_testlib import K8

pytestmark = pytest.mark.gpu


class Pool:
    def __init__(self, lens, spare, cols, seed=0, capacity=None, held=None):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        self.nr = len(lens)
        self.held = -(-np.maximum(self.lens, 0) // 16) if held is None else np.asarray(held)
        self.held = self.held.astype(np.int32)
        ids = rng.permutation(int(self.held.sum()) + spare + 7).astype(np.int32)
        self.table, at = np.full((self.nr, cols), -1, np.int32), 0
        for r, h in enumerate(np.minimum(self.held, cols)):
            self.table[r, :h] = ids[at:at + h]
            at += h
        self.free = np.full(capacity or ids.size, -5, np.int32)
        self.free[:spare] = ids[at:at + spare]
        self.count = spare
        g = lambda a: torch.as_tensor(a).cuda()  # noqa: E731
        self.t_table, self.t_held, self.t_free = g(self.table), g(self.held), g(self.free)
        self.t_count, self.t_lens = torch.tensor([spare], dtype=torch.int32, device="cuda"), g(self.lens)
        self.ws = s3r.new_workspace(s3r.s3r_pages_workspace_size(self.nr))

    def batch(self, ids=None):
        return s3r.make_batch(self.t_lens, self.t_table, req_ids=None if ids is None else torch.tensor(ids, dtype=torch.int32, device="cuda"))

    def alloc(self, T, n_new=None, ids=None, in_place=False, slots=True):
        ho = self.t_held if in_place else torch.full_like(self.t_held, -7)
        co = self.t_count if in_place else torch.full_like(self.t_count, -7)
        granted = torch.full_like(self.t_held, -7)
        sm = torch.full((self.nr, T), -9, dtype=torch.int64, device="cuda") if slots else None
        s3r.s3r_alloc_pages(self.batch(ids), T, self.t_held, self.t_free, self.t_count, ho, co, granted, self.ws,
                            n_new=None if n_new is None else torch.as_tensor(np.asarray(n_new, dtype=np.int32)).cuda(), slot_map=sm)
        return [x if x is None else x.cpu().numpy() for x in (self.t_table, ho, co, granted, sm)]

    def check_alloc(self, got, T, n_new=None, ids=None):
        n = np.full(self.nr, T) if n_new is None else np.asarray(n_new)
        t, h, c, g, sl = K8.alloc_pages(self.table, self.lens, n, T, self.held, self.free, self.count, ids)
        np.testing.assert_array_equal(got[0], t)
        sel = slice(None) if ids is None else list(ids)
        np.testing.assert_array_equal(got[1][sel], h[sel])
        assert got[2].tolist() == [c]
        np.testing.assert_array_equal(got[3][sel], g[sel])
        if got[4] is not None:
            np.testing.assert_array_equal(got[4][sel], sl[sel])
            if ids is not None:
                rest = sorted(set(range(self.nr)) - set(ids))
                assert (got[4][rest] == -9).all() and (got[1][rest] == -7).all() and (got[3][rest] == -7).all()
        return t, h, c, g


@pytest.mark.parametrize("lens,T,spare", [
    ([0], 1, 1), ([15, 16, 17], 1, 5), ([100, 0, 5, 31], 7, 6),
    ([0] * 5, 100, 35),                       # exactly what is asked for
    ([0] * 5, 100, 34),                       # one page short: the last request gets none
    ([0, 3, 9], 5000, 2000), ([7] * 700, 7, 500),
    ([0] * 300, 17, 1000), ([0, 40000], 9000, 2000),
])
def test_alloc_matches_oracle(lens, T, spare):
    cols = -(-(max(lens) + T) // 16)
    p = Pool(lens, spare, cols)
    p.check_alloc(p.alloc(T), T)
    assert s3r.s3r_get_error(p.ws) == 0


def test_alloc_ragged_subset_in_place_and_again():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 500, size=90)
    n = rng.integers(0, 61, size=90)
    p = Pool(lens, 200, 64, seed=4)
    ids = rng.permutation(90)[:50].tolist()
    t, h, c, g = p.check_alloc(p.alloc(60, n, ids, slots=False), 60, n, ids)
    # (the call above wrote its counts elsewhere, so the same call in place gives the same)
    got = p.alloc(60, n, ids, in_place=True)
    np.testing.assert_array_equal(got[0], t)
    np.testing.assert_array_equal(p.t_held.cpu().numpy(), h)
    assert p.t_count.tolist() == [c]
    again = p.alloc(60, n, ids, in_place=True)             # everything that was served is held now
    np.testing.assert_array_equal(again[1], h)
    served = [r for r in ids if g[r]]
    np.testing.assert_array_equal(again[4][served], got[4][served])
    assert s3r.s3r_get_error(p.ws) == 0


@pytest.mark.parametrize("T", [511, 512, 513, 601, 4097, 8193])
def test_alloc_long_slot_maps_of_odd_length(T):
    """Slot rows that start at either half of 16 bytes, ragged, in segments of one to several CTAs; ids
    out of order, and requests that the stack has no pages for."""
    rng = np.random.default_rng(T)
    lens, n = rng.integers(0, 40, size=9), rng.integers(0, T + 1, size=9)
    n[2], n[5] = 0, T
    p = Pool(lens, int(5 * T / 16), -(-(40 + T) // 16), seed=T)
    ids = rng.permutation(9)[:7].tolist()
    p.check_alloc(p.alloc(T, n, ids), T, n, ids)
    p.check_alloc(p.alloc(T, n), T, n)
    assert s3r.s3r_get_error(p.ws) == 0


def test_alloc_reports_what_is_out_of_range():
    p = Pool([10, -3, 20, 30, 40], 10, 4, held=[1, 0, 2, 2, 9])
    n = np.array([5, 5, 61, 40, 3])     # 1: negative length; 2: more than T; 3: past four pages; 4: holds too many
    got = p.alloc(60, n)
    assert s3r.s3r_get_error(p.ws) == 1 << 5
    p.check_alloc(got, 60, n)
    assert got[3].tolist() == [1, 0, 0, 0, 0]
    p.t_count.fill_(p.free.size + 1)    # a stack count past its array
    got = p.alloc(5)
    assert s3r.s3r_get_error(p.ws) == 1 << 5 and got[0].tolist() == p.table.tolist()
    q = Pool([10, 20], 10, 4)
    got = q.alloc(30, ids=[1, 2])       # an id out of range
    assert s3r.s3r_get_error(q.ws) == 1 << 5 and got[3][1] == 1


@pytest.mark.parametrize("lens,keep,cols", [
    ([16381], 0, 1024), ([100, 0, 5, 31], 16, 8), ([500] * 300, 100, 40), ([40000, 1, 3000], 33, 2500), ([7] * 700, 0, 1),
])
def test_release_matches_oracle_in_and_out_of_place(lens, keep, cols):
    p = Pool(lens, 13, cols, seed=2)
    k = np.minimum(np.full(p.nr, keep), np.asarray(lens)).astype(np.int32)
    f, h, c = K8.release_pages(p.table, k, p.held, p.free, p.count)
    for in_place in (False, True):
        ho = p.t_held if in_place else torch.full_like(p.t_held, -7)
        co = p.t_count if in_place else torch.full_like(p.t_count, -7)
        s3r.s3r_release_pages(p.batch(), p.t_held, p.t_free, p.t_count, ho, co, p.ws,
                              keep_len=torch.as_tensor(k).cuda() if keep else None)
        assert s3r.s3r_get_error(p.ws) == 0
        np.testing.assert_array_equal(p.t_free.cpu().numpy(), f)
        np.testing.assert_array_equal(ho.cpu().numpy(), h)
        assert co.tolist() == [c]
        np.testing.assert_array_equal(p.t_table.cpu().numpy(), p.table)


def test_release_keeps_what_does_not_fit():
    p = Pool([160, 160, 160], 5, 10, capacity=26)          # room for 21 pages, 30 held
    k = np.array([0, 0, 0], np.int32)
    ho, co = torch.empty_like(p.t_held), torch.empty_like(p.t_count)
    s3r.s3r_release_pages(p.batch(), p.t_held, p.t_free, p.t_count, ho, co, p.ws)
    assert s3r.s3r_get_error(p.ws) == 1 << 5
    f, h, c = K8.release_pages(p.table, k, p.held, p.free, p.count)
    assert h.tolist() == [0, 0, 10] and c == 25
    np.testing.assert_array_equal(p.t_free.cpu().numpy(), f)
    assert ho.tolist() == h.tolist() and co.tolist() == [c]


def test_pages_come_back_and_go_out_again():
    """A serving loop: requests grow, end and are admitted again; no page is lost or held twice."""
    rng = np.random.default_rng(8)
    nr, total = 20, 400
    p = Pool([0] * nr, total, 64)
    lens = np.zeros(nr, dtype=np.int64)
    granted = torch.zeros(nr, dtype=torch.int32, device="cuda")
    for it in range(30):
        n = rng.integers(0, 40, size=nr).astype(np.int32)
        s3r.s3r_alloc_pages(p.batch(), 40, p.t_held, p.t_free, p.t_count, p.t_held, p.t_count, granted, p.ws, n_new=torch.as_tensor(n).cuda())
        lens += np.where(granted.cpu().numpy() == 1, n, 0)
        done = rng.random(nr) < 0.15
        lens[done] = 0
        p.t_lens.copy_(torch.as_tensor(lens.astype(np.int32)))
        s3r.s3r_release_pages(p.batch(), p.t_held, p.t_free, p.t_count, p.t_held, p.t_count, p.ws, keep_len=p.t_lens)
        held, table, count = p.t_held.cpu().numpy(), p.t_table.cpu().numpy(), int(p.t_count)
        np.testing.assert_array_equal(held, -(-lens // 16))
        out = np.concatenate([table[r, :h] for r, h in enumerate(held)] + [p.t_free.cpu().numpy()[:count]])
        assert sorted(out.tolist()) == sorted(p.free[:total].tolist())
    assert s3r.s3r_get_error(p.ws) == 0
