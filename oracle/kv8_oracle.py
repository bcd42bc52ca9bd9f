"""Oracle of the 8-bit cache and of the page calls (numpy).

e4m3 (OCP FP8): 1 sign, 4 exponent (bias 7), 3 mantissa bits; no infinities, code 0x7f / 0xff is
NaN, largest value 448. A page's scale is 2^e, e the least integer >= -126 with
max |x| <= 448 * 2^e over the page's live rows of one KV head (1 if all are zero)."""
from __future__ import annotations

import math

import numpy as np

PAGE = 16
MAX = 448.0


def _decode(c):
    s, e, m = c >> 7, (c >> 3) & 15, c & 7
    if e == 15 and m == 7:
        return math.nan
    v = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
    return -v if s else v


E4M3 = np.array([_decode(c) for c in range(256)])


def encode(x):
    """Codes (uint8) of finite x, |x| <= 448 after rounding: nearest, ties to the even code."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.abs(x)
    grid = E4M3[:127]                                       # 0 .. 448 ascending
    hi = np.clip(np.searchsorted(grid, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - grid[lo], grid[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return np.where(np.signbit(x), code | 0x80, code).astype(np.uint8)


def page_scale(amax: float) -> float:
    if amax == 0:
        return 1.0
    e = -126
    while amax > MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append_request(codes, scale, pages, start, rows):
    """In place: rows [n][H][d] (float) of one request at positions start.. into codes
    [P][H][16][d] uint8 / scale [P][H] float32, pages its page-table row."""
    n, H, _ = rows.shape
    end = start + n
    for pg in range(start // PAGE, -(-end // PAGE) if n else start // PAGE):
        lo, hi = pg * PAGE, min((pg + 1) * PAGE, end)
        first = max(lo, start)
        if first >= hi:
            continue
        for h in range(H):
            old = np.float32(E4M3[codes[pages[pg], h, : first - lo]]) * np.float32(scale[pages[pg], h])
            x = np.concatenate([old.astype(np.float32), rows[first - start: hi - start, h].astype(np.float32)])
            x = np.where(np.isfinite(x), x, np.float32(0))
            s = page_scale(float(np.abs(x).max()))
            codes[pages[pg], h, : hi - lo] = encode(np.float64(x) / s)
            scale[pages[pg], h] = s


def dequantise(codes, scale, pages, upto):
    """[H][upto][d] float64 values of positions 0..upto-1."""
    pages = np.asarray(pages)[: -(-upto // PAGE)]
    x = E4M3[codes[pages]] * scale[pages].astype(np.float64)[:, :, None, None]
    return x.transpose(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :upto]


def alloc_pages(table, lens, n_new, T, held, free, count, ids=None):
    """(table, held, count, granted, slots) after an allocation, requests in batch order."""
    nr, cols = table.shape
    table, held_out = table.copy(), held.copy()
    granted, slots = np.zeros(nr, np.int32), np.full((nr, T), -1, np.int64)
    asked = taken = 0
    for r in (range(nr) if ids is None else ids):
        L, n, h = int(lens[r]), int(n_new[r]), int(held[r])
        need = -(-(L + n) // PAGE)
        if L < 0 or not 0 <= n <= T or not 0 <= h <= cols or need > cols:
            continue
        add = max(0, need - h)
        before, asked = asked, asked + add
        if add and asked > count:
            continue
        for i in range(add):
            table[r, h + i] = free[count - 1 - before - i]
        held_out[r], granted[r], taken = h + add, 1, taken + add
        for t in range(n):
            slots[r, t] = int(table[r, (L + t) // PAGE]) * PAGE + (L + t) % PAGE
    return table, held_out, count - taken, granted, slots


def release_pages(table, keep_len, held, free, count, ids=None):
    """(free, held, count) after a release, requests in batch order."""
    free, held_out = free.copy(), held.copy()
    nr, cols = table.shape
    asked = taken = 0
    for r in (range(nr) if ids is None else ids):
        h, k = int(held[r]), int(keep_len[r])
        if k < 0 or not 0 <= h <= cols:
            continue
        keep = -(-k // PAGE)
        gone = max(0, h - keep)
        before, asked = asked, asked + gone
        if gone and count + asked > free.size:
            continue
        free[count + before: count + before + gone] = table[r, keep:h]
        held_out[r], taken = h - gone, taken + gone
    return free, held_out, count + taken
