"""Shared helpers of the 8-bit cache's tests: seeded caches on the device, their 64-bit values,
and the error bounds of the attention calls, derived from the roundings the kernels make."""
from __future__ import annotations

import math

import numpy as np
import torch

import sparse_dense_kv_b200 as s3r
from oracle import kv8_oracle as K8
from oracle import s3r_oracle as O


class KV8Case:
    """Requests of committed lengths `lens` with room for `extra` tokens, all slots filled with
    codes of normal values; slots behind `upto` (default: the room's end) hold NaN codes."""

    def __init__(self, Hkv, d, lens, extra, seed=0, shuffle=True, std=60.0, pow2=True, scale_spread=3, upto=None):
        rng = np.random.default_rng(seed)
        self.Hkv, self.d, self.lens = Hkv, d, np.asarray(lens, dtype=np.int64)
        pages = -(-(self.lens + extra) // 16)
        self.total, self.max_pages, self.nr = max(1, int(pages.sum())), max(1, int(pages.max())), len(lens)
        ids = rng.permutation(self.total) if shuffle else np.arange(self.total)
        self.pt = np.full((self.nr, self.max_pages), -1, dtype=np.int32)
        at = 0
        for r, n in enumerate(pages):
            self.pt[r, :n] = ids[at:at + n]
            at += n
        shape = (self.total, Hkv, 16, d)
        g = torch.Generator().manual_seed(seed)
        enc = lambda: (torch.randn(shape, generator=g) * std).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        self.kc, self.vc = enc(), enc()
        e = rng.integers(-7 - scale_spread, -6, size=(2, self.total, Hkv))
        sc = np.exp2(e.astype(np.float64)) * (1.0 if pow2 else rng.uniform(0.6, 1.4, size=e.shape))
        self.ks, self.vs = torch.as_tensor(sc[0].astype(np.float32)), torch.as_tensor(sc[1].astype(np.float32))
        for r in range(self.nr):   # what lies behind the last token is whatever was there
            end = int(self.lens[r] + (extra if upto is None else upto))
            if end % 16:
                self.kc[self.pt[r, end // 16], :, end % 16:] = 0x7F
                self.vc[self.pt[r, end // 16], :, end % 16:] = 0xFF

    def cuda(self, Hq, workspace_k=8, sel_stride=1):
        self.k, self.v, self.k_scale, self.v_scale = (t.cuda() for t in (self.kc, self.vc, self.ks, self.vs))
        self.page_table = torch.as_tensor(self.pt).cuda()
        self.seq_lens = torch.as_tensor(self.lens.astype(np.int32)).cuda()
        self.cache = s3r.make_kv8_cache(self.k, self.v, self.k_scale, self.v_scale, Hq)
        self.batch = s3r.make_batch(self.seq_lens, self.page_table)
        self.ws = s3r.new_workspace(s3r.s3r_kv8_workspace_size(self.cache, self.nr, self.max_pages, workspace_k, 64, sel_stride))
        return self

    def values(self, r, upto):
        """K, V [Hkv][upto][d] float64 of request r from the device's pools."""
        return (K8.dequantise(c.view(torch.uint8).cpu().numpy(), s.cpu().numpy(), self.pt[r], upto)
                for c, s in ((self.k, self.k_scale), (self.v, self.v_scale)))


def logit_bound(q, K, split):
    """Per (row, position) bound on a logit's error, [H][R][n]: q [H][R][d], K [H][n][d]. `split`:
    the absolute error of an element of q relative to the row's largest (2^-18 for two e4m3
    parts, 2^-31 for a half). The products and sums are fp32: the tensor core adds at least 24-bit
    products in groups, so 2^-20 of the sum of magnitudes covers its roundings and the two
    multiplications (page scale, row factor) behind it."""
    d = q.shape[-1]
    a = np.abs(K)
    qm = np.abs(q).max(-1, keepdims=True)
    sums = np.einsum("hrd,hnd->hrn", np.abs(q), a)
    return (2.0 ** -20 * sums + split * qm * a.sum(-1)[:, None, :]) / math.sqrt(d)


def attention_bounds(q, K, V, vis, split, p_step):
    """64-bit attention of rows q [H][R][d] over K, V [H][n][d] with vis [R][n] and the bounds of
    the kernel's out, lse and logits: (out, lse, x, b_out, b_lse, b_x).

    With e the largest logit error of a row (plus 2^-21 for 2^x and the maximum's rounding, and
    2^-22 of the largest |logit|): weights are off by a factor e^(+-2e), so out by 2e sum p|v|;
    P's rounding adds p_step sum p|v|; the output is rounded to bf16 once (2^-8 of it)."""
    x = np.einsum("hrd,hnd->hrn", q, K) / math.sqrt(q.shape[-1])
    bx = logit_bound(q, K, split) + 2.0 ** -22 * np.abs(x)
    xm = np.where(vis[None], x, -np.inf)
    m = xm.max(-1, keepdims=True)
    p = np.exp(xm - m)
    z = p.sum(-1, keepdims=True)
    p /= z
    out, lse = p @ V, (m + np.log(z))[..., 0]
    e = np.where(vis[None], bx, 0).max(-1) + 2.0 ** -21 + 2.0 ** -22 * np.abs(m[..., 0])
    pv = p @ np.abs(V)
    b_out = 2.0 ** -8 * np.abs(out) + (2 * e[..., None] + p_step + 2.0 ** -18) * pv + 1e-30
    return out, lse, x, b_out, e + 2.0 ** -21 * (1 + np.abs(lse)), bx


def rows_of(q, Hkv):
    """[T][Hq][d] -> [Hkv][T*G][d] (row t*G + g)."""
    T, Hq, d = q.shape
    return q.reshape(T, Hkv, Hq // Hkv, d).transpose(1, 0, 2, 3).reshape(Hkv, -1, d)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def assert_within(got, want, bound, what):
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(err / bound):.3g} x the bound, max err {np.nanmax(err):.3g}"


# P's rounding: two e4m3 parts and the half between them (verify), or a half (draft)
VERIFY = dict(split=2.0 ** -18, p_step=2.0 ** -8)
DRAFT = dict(split=2.0 ** -31, p_step=2.0 ** -10)
__all__ = ["KV8Case", "attention_bounds", "rows_of", "f64", "assert_within", "VERIFY", "DRAFT", "K8", "O"]
