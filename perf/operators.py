"""Cases of the 8-bit KV cache's operators: what a rollout server calls on a paged cache whose
keys and values are held in e4m3 with one scale per (page of 16 positions, KV head).

  alloc    s3r_alloc_pages            pages and slots for the next tokens of every request
  release  s3r_release_pages          finished requests give their pages back
  append   s3r_kv8_append             bf16 rows into the 8-bit pages, with their scales
  verify   s3r_verify_attn_kv8        dense attention of k + 1 block rows over the 8-bit cache
  draft    s3r_sparse_draft_attn_kv8  attention of one draft row over a selected set

With `own` false, run() computes the operator in its plain form from elementary torch operations
in 32 bits; with `own` true it makes the library's calls. exact() computes the attention and the
quantisation in 64 bits from their definitions, request by request. A float8 tensor is returned
as it is (its elements are values), beside the scales that multiply it.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
F8 = torch.float8_e4m3fn
F8_MAX = 448.0


# --------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new request of a small model decodes its first tokens: nothing but latency
        dict(name="verify-one-row-short", op="verify", nr=1, hq=16, hkv=8, d=128, k=0, lo=77, hi=77, capture=False, shuffle=False, pattern=1),
        # the benchmark's workload: 32 requests of 8K to 24K tokens, 6 drafts, logits captured for the next selection
        dict(name="verify-32x8k-24k-k6", op="verify", nr=32, hq=32, hkv=8, d=128, k=6, lo=8192, hi=24576, capture=True, shuffle=False, pattern=2),
        # a ragged batch over scattered pages, two query heads per KV head, no capture (plain decoding of a block)
        dict(name="verify-96-ragged-scattered", op="verify", nr=96, hq=16, hkv=8, d=128, k=6, lo=1024, hi=16384, capture=False, shuffle=True, pattern=3),
        # the smallest workload of the tests: two short requests, head_dim 64
        dict(name="draft-tiny-d64", op="draft", nr=2, hq=2, hkv=1, d=64, lo=256, hi=300, budget=2500, window=16, shuffle=False, pattern=4),
        # one draft step of the benchmark's workload, 5 % of the cache
        dict(name="draft-32x8k-24k-5pct", op="draft", nr=32, hq=32, hkv=8, d=128, lo=8192, hi=24576, budget=500, window=64, shuffle=False, pattern=5),
        # the budget sweep's largest set: 20 % of 24K tokens
        dict(name="draft-32x24k-20pct", op="draft", nr=32, hq=32, hkv=8, d=128, lo=24576, hi=24576, budget=2000, window=64, shuffle=True, pattern=6),
        # the k + 1 rows of a round enter the cache at odd positions
        dict(name="append-round-32x7", op="append", nr=32, hkv=8, d=128, lo=8192, hi=24576, t=7, ragged=False, shuffle=False, pattern=7),
        # ragged prompts of up to 8K tokens are written after their prefill
        dict(name="append-prompts-16x8k", op="append", nr=16, hkv=8, d=128, lo=0, hi=0, t=8191, ragged=True, shuffle=True, pattern=8),
        # every round: room for k + 1 tokens of 32 requests
        dict(name="alloc-round-32x7", op="alloc", nr=32, lo=8192, hi=24576, t=7, ragged=False, pattern=9),
        # 256 ragged prompts are admitted at once
        dict(name="alloc-prompts-256x16k", op="alloc", nr=256, lo=0, hi=0, t=16384, ragged=True, pattern=10),
        # one long request ends
        dict(name="release-one", op="release", nr=1, lo=16381, hi=16381, pattern=11),
        # a whole ragged batch ends, each request keeping its shared prompt
        dict(name="release-256-ragged", op="release", nr=256, lo=1024, hi=16384, pattern=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["verify", "verify", "draft", "draft", "append", "append", "alloc", "release"])
    c = dict(op=op, pattern=rng.randrange(1, 1 << 30))
    if op in ("verify", "draft"):
        hq, hkv, d = rng.choice([(32, 8, 128), (16, 8, 128), (8, 1, 128), (64, 8, 128), (2, 1, 64), (12, 4, 64), (6, 2, 128), (4, 4, 128)])
        nr, hi = _log(rng, 1, 64), _log(rng, 1, 24576)
        while nr * hi * hkv > 32 * 16384 * 4:
            nr, hi = max(1, nr // 2), max(1, hi * 3 // 4)
        lo = rng.choice([hi, max(0, hi // 3), 0])
        c.update(nr=nr, hq=hq, hkv=hkv, d=d, lo=lo, hi=hi, shuffle=rng.random() < 0.5)
        if op == "verify":
            c.update(k=rng.randrange(0, min(8, 64 // (hq // hkv) - 1) + 1), capture=rng.random() < 0.5)
        else:
            c.update(budget=rng.choice([1, 200, 500, 1000, 2000, 10000]), window=rng.choice([1, 16, 64, 200]))
            if c["budget"] == 10000:
                c["hi"], c["lo"] = min(c["hi"], 4096), min(c["lo"], 4096)
    elif op == "append":
        hkv, d = rng.choice([(8, 128), (1, 64), (4, 64), (2, 128), (1, 128)])
        t, nr = _log(rng, 1, 8192), _log(rng, 1, 128)
        while nr * t * hkv > 16 * 8191 * 4:
            nr, t = max(1, nr // 2), max(1, t * 3 // 4)
        hi = rng.choice([0, 15, 333, 4000])
        c.update(nr=nr, hkv=hkv, d=d, lo=hi // 2, hi=hi, t=t, ragged=rng.random() < 0.5, shuffle=rng.random() < 0.5)
    elif op == "alloc":
        t, nr = _log(rng, 1, 16384), _log(rng, 1, 1000)
        while nr * t > 256 * 16384 // 2:
            nr, t = max(1, nr // 2), max(1, t * 3 // 4)
        hi = rng.choice([0, 100, 5000])
        c.update(nr=nr, lo=hi // 2, hi=hi, t=t, ragged=rng.random() < 0.5)
    else:
        nr, hi = _log(rng, 1, 1000), _log(rng, 1, 16384)
        while nr * hi > 256 * 16384 // 2:
            nr, hi = max(1, nr // 2), max(1, hi * 3 // 4)
        c.update(nr=nr, lo=hi // 4, hi=hi)
    return c


def _lengths(case):
    """Committed lengths of the case's requests: log-uniform in [lo, hi], the case's own."""
    r = np.random.default_rng([case["pattern"], 1])
    lo, hi = case["lo"], case["hi"]
    x = np.exp(r.uniform(math.log(lo + 1), math.log(hi + 1), size=case["nr"])) - 1
    if case["op"] in ("verify", "draft", "append") and lo * 4 > hi:   # the benchmark's are uniform
        x = r.uniform(lo, hi, size=case["nr"])
    return np.clip(np.round(x), lo, hi).astype(np.int64)


def _new_counts(case):
    r = np.random.default_rng([case["pattern"], 2])
    n = np.full(case["nr"], case["t"], dtype=np.int64)
    if case["ragged"]:
        n = np.minimum(np.round(np.exp(r.uniform(0.0, math.log(case["t"] + 1), size=case["nr"]))), case["t"]).astype(np.int64)
        n[0] = case["t"]
    return n


def _steps(case):
    return np.random.default_rng([case["pattern"], 3]).integers(0, 6, size=case["nr"])


def _set_sizes(case, lens):
    w = np.minimum(case["window"], lens)
    n = -(-(lens * case["budget"]) // 10000)
    return np.minimum(np.maximum(n, w), lens), w


def work(case):
    lens = _lengths(case)
    op, nr = case["op"], case["nr"]
    if op == "verify":
        T, G, H, d = case["k"] + 1, case["hq"] // case["hkv"], case["hkv"], case["d"]
        end = lens + T
        bytes_ = int(end.sum()) * H * d * 2 + int((-(-end // PAGE)).sum()) * (H * 8 + 4)
        bytes_ += nr * T * case["hq"] * (d * 4 + 4) + 4 * nr
        if case["capture"]:
            bytes_ += int(lens.sum()) * H * G * T * 4
        seen = int((lens * T).sum()) + nr * T * (T + 1) // 2
        return {"bytes": bytes_, "flops": 4 * seen * case["hq"] * d}
    if op == "draft":
        n, _ = _set_sizes(case, lens)
        a = n + _steps(case) + 1
        rows = int(a.sum()) * case["hkv"]
        bytes_ = rows * case["d"] * 2 + int(n.sum()) * case["hkv"] * 4 + nr * case["hq"] * (case["d"] * 4 + 4)
        return {"bytes": bytes_, "flops": 4 * int(a.sum()) * case["hq"] * case["d"]}
    if op == "append":
        n = int(_new_counts(case).sum())
        return {"bytes": n * case["hkv"] * case["d"] * 2 * 3 + (n // PAGE + 2 * nr) * (case["hkv"] * 8 + 4), "flops": n * case["hkv"] * case["d"] * 2 * 4}
    if op == "alloc":
        n = _new_counts(case)
        add = -(-(lens + n) // PAGE) - -(-lens // PAGE)
        return {"bytes": int(add.sum()) * 8 + nr * case["t"] * 8 + nr * 24, "flops": nr * 8}
    held = -(-lens // PAGE)
    return {"bytes": int((held - -(-(lens // 3) // PAGE)).sum()) * 8 + nr * 16, "flops": nr * 4}


# --------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 12345)
    return g


def _table(case, tokens, seed):
    """Page table [nr][max pages] of requests that hold pages for `tokens` positions each."""
    r = np.random.default_rng([int(seed), 4])
    pages = -(-tokens // PAGE)
    total = max(1, int(pages.sum()))
    ids = r.permutation(total) if case.get("shuffle") else np.arange(total)
    pt = np.full((case["nr"], max(1, int(pages.max()))), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(pages):
        pt[i, :n] = ids[at:at + n]
        at += n
    return torch.as_tensor(pt).cuda(), total


def _cache(case, pt, total, tokens, seed, garbage=True):
    """8-bit pools and scales: normal values with a few large keys, each page and head with a
    scale of its own; slots behind a request's last token hold whatever was there (NaN)."""
    g = _gen(seed)
    H, d = case["hkv"], case["d"]

    def pool(large):
        out = torch.empty((total, H, PAGE, d), dtype=F8, device="cuda")
        for a in range(0, total, 4096):
            x = torch.randn((min(4096, total - a), H, PAGE, d), generator=g, device="cuda") * 50.0
            if large:
                pick = torch.rand(x.shape[:3], generator=g, device="cuda") < 0.002
                x = torch.where(pick[..., None], x * 4.0, x)
            out[a:a + 4096] = x.clamp_(-F8_MAX, F8_MAX).to(F8)
        return out

    k_pool, v_pool = pool(True), pool(False)
    sc = [torch.exp2(torch.randint(-7, -4, (total, H), generator=g, device="cuda").float()) for _ in range(2)]
    if garbage:
        last = np.maximum(tokens - 1, 0) // PAGE
        page = pt[torch.arange(case["nr"], device="cuda"), torch.as_tensor(last).cuda()].long().clamp_min(0)
        used = torch.as_tensor(tokens - last * PAGE).cuda()
        behind = torch.arange(PAGE, device="cuda")[None, :] >= used[:, None]
        for p in (k_pool, v_pool):
            u = p.view(torch.uint8)
            u[page] = torch.where(behind[:, None, :, None], torch.full_like(u[page], 0x7F), u[page])
    return dict(k_pool=k_pool, v_pool=v_pool, k_scale=sc[0], v_scale=sc[1])


def prepare(case, seed):
    lens = _lengths(case)
    nr, op = case["nr"], case["op"]
    g = _gen(seed + 17)
    dev = dict(device="cuda")
    s = dict(op=op, case=case, seq_lens=torch.as_tensor(lens, dtype=torch.int32).cuda())
    if op == "verify":
        T = case["k"] + 1
        pt, total = _table(case, lens + T, seed)
        s.update(_cache(case, pt, total, lens + T, seed), page_table=pt, T=T)
        s["q"] = torch.randn((nr, T, case["hq"], case["d"]), generator=g, **dev).to(torch.bfloat16)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((nr, T, case["hq"]), **dev)
        s["scores"] = None
        if case["capture"]:
            s["scores"] = torch.zeros((nr, case["hkv"], case["hq"] // case["hkv"] * T, pt.shape[1] * PAGE), **dev)
    elif op == "draft":
        steps = _steps(case)
        pt, total = _table(case, lens + steps + 1, seed)
        s.update(_cache(case, pt, total, lens + steps + 1, seed), page_table=pt)
        s["step"] = torch.as_tensor(steps, dtype=torch.int32).cuda()
        s["q"] = torch.randn((nr, case["hq"], case["d"]), generator=g, **dev).to(torch.bfloat16)
        n, w = _set_sizes(case, lens)
        idx = torch.zeros((nr, case["hkv"], max(1, int(n.max()))), dtype=torch.int32, **dev)
        for r in range(nr):
            L, a = int(lens[r]), int(n[r] - w[r])
            old = torch.rand((case["hkv"], max(1, L - int(w[r]))), generator=g, **dev).topk(a, dim=1).indices.sort(dim=1).values
            new = torch.arange(L - int(w[r]), L, **dev).expand(case["hkv"], -1)
            idx[r, :, : int(n[r])] = torch.cat([old, new], dim=1).int()
        s["sel_idx"], s["sel_count"] = idx, torch.as_tensor(np.repeat(n[:, None], case["hkv"], 1), dtype=torch.int32).cuda()
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((nr, case["hq"]), **dev)
    elif op == "append":
        n = _new_counts(case)
        pt, total = _table(case, lens + n, seed)
        s.update(_cache(case, pt, total, lens + n, seed, garbage=False), page_table=pt, T=case["t"])
        s["n_new"] = torch.as_tensor(n, dtype=torch.int32).cuda()
        shape = (nr, case["t"], case["hkv"], case["d"])
        mag = torch.exp2(torch.randint(-2, 3, (nr, case["t"], 1, 1), generator=g, **dev).float())
        s["k_new"] = (torch.randn(shape, generator=g, **dev) * mag).to(torch.bfloat16)
        s["v_new"] = torch.randn(shape, generator=g, **dev).to(torch.bfloat16)
    else:
        r = np.random.default_rng([int(seed), 5])
        held = -(-lens // PAGE)
        if op == "alloc":
            n = _new_counts(case)
            need = -(-(lens + n) // PAGE)
            spare = int((need - held).sum()) + 64
            cols = max(1, int(need.max()))
            s.update(n_new=torch.as_tensor(n, dtype=torch.int32).cuda(), T=case["t"])
        else:
            spare, cols = 1000, max(1, int(held.max()))
            s["keep_len"] = torch.as_tensor(lens // 3, dtype=torch.int32).cuda()
        ids = r.permutation(int(held.sum()) + spare).astype(np.int32)
        pt, at = np.full((nr, cols), -1, dtype=np.int32), 0
        for i, h in enumerate(held):
            pt[i, :h] = ids[at:at + h]
            at += h
        free = np.full(ids.size, -1, dtype=np.int32)
        free[:spare] = ids[at:]
        s.update(page_table=torch.as_tensor(pt).cuda(), held=torch.as_tensor(held, dtype=torch.int32).cuda(),
                 free_pages=torch.as_tensor(free).cuda(), free_count=torch.tensor([spare], dtype=torch.int32, **dev))
        s.update(held_out=torch.zeros(nr, dtype=torch.int32, **dev), free_count_out=torch.zeros(1, dtype=torch.int32, **dev))
        if op == "alloc":
            s.update(granted=torch.zeros(nr, dtype=torch.int32, **dev), slots=torch.zeros((nr, case["t"]), dtype=torch.int64, **dev))
    return s


# --------------------------------------------------------------------------------- passes
def run(s):
    if own:
        return _own(s)
    return {"verify": _plain_verify, "draft": _plain_draft, "append": _plain_append, "alloc": _plain_alloc, "release": _plain_release}[s["op"]](s)


def _handles(s):
    """The descriptors and the workspace that a program makes once and keeps."""
    import sparse_dense_kv_b200 as s3r
    h = dict(s3r=s3r, batch=s3r.make_batch(s["seq_lens"], s["page_table"]))
    nr, pages = s["page_table"].shape
    if "k_pool" in s:
        h["cache"] = s3r.make_kv8_cache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["case"].get("hq", s["case"]["hkv"]))
        stride = s["sel_idx"].shape[-1] if "sel_idx" in s else 1
        n = s3r.s3r_kv8_workspace_size(h["cache"], nr, pages, s["case"].get("k", 0), 1, stride)
    else:
        n = s3r.s3r_pages_workspace_size(nr)
    h["ws"] = s3r.new_workspace(n)
    return h


def _own(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    h = s["handles"]
    s3r, ws, batch = h["s3r"], h["ws"], h["batch"]
    if s["op"] == "verify":
        s3r.s3r_verify_attn_kv8(h["cache"], batch, s["T"] - 1, s["q"], s["out"], s["lse"], s["scores"], ws)
        return dict(out=s["out"], lse=s["lse"], scores=s["scores"])
    if s["op"] == "draft":
        s3r.s3r_sparse_draft_attn_kv8(h["cache"], batch, s["step"], s["q"], s["sel_idx"], s["sel_count"], s["out"], s["lse"], ws)
        return dict(out=s["out"], lse=s["lse"])
    if s["op"] == "append":
        s3r.s3r_kv8_append(h["cache"], batch, s["k_new"], s["v_new"], ws, n_new=s["n_new"])
        return dict(k=s["k_pool"], v=s["v_pool"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["op"] == "alloc":
        s3r.s3r_alloc_pages(batch, s["T"], s["held"], s["free_pages"], s["free_count"], s["held_out"], s["free_count_out"], s["granted"], ws,
                            n_new=s["n_new"], slot_map=s["slots"])
        return dict(table=s["page_table"], held=s["held_out"], count=s["free_count_out"], granted=s["granted"], slots=s["slots"])
    s3r.s3r_release_pages(batch, s["held"], s["free_pages"], s["free_count"], s["held_out"], s["free_count_out"], ws, keep_len=s["keep_len"])
    return dict(free=s["free_pages"], held=s["held_out"], count=s["free_count_out"])


def _rows(pool, scale, page, head, slot):
    """Dequantised rows [..., d] in 32 bits at the given (page, head, slot) indices."""
    return pool.view(torch.uint8)[page, head, slot].view(F8).float() * scale[page, head].unsqueeze(-1)


def _plain_verify(s):
    c, T, pt = s["case"], s["T"], s["page_table"]
    H, d, G, nr = c["hkv"], c["d"], c["hq"] // c["hkv"], c["nr"]
    cap = pt.shape[1] * PAGE
    L = s["seq_lens"].long().view(nr, 1, 1, 1)
    page = pt.long().clamp_min(0)
    pos = torch.arange(cap, device="cuda")
    inside = (pos < L[:, :, :, 0] + T).view(nr, 1, cap, 1)

    def dense(pool, scale):
        x = pool.view(torch.uint8)[page].view(F8).float() * scale[page][..., None, None]      # [nr][pages][H][16][d]
        x = x.permute(0, 2, 1, 3, 4).reshape(nr, H, cap, d)
        return torch.where(inside, x, torch.zeros((), device="cuda"))

    q = s["q"].float().view(nr, T, H, G, d).permute(0, 2, 1, 3, 4).reshape(nr, H, T * G, d)
    x = q @ dense(s["k_pool"], s["k_scale"]).transpose(2, 3) * (1.0 / math.sqrt(d))            # [nr][H][T*G][cap]
    t = (torch.arange(T * G, device="cuda") // G).view(1, 1, T * G, 1)
    if s["scores"] is not None:
        s["scores"].copy_(torch.where(pos < L, x, s["scores"]))
    x = torch.where(pos <= L + t, x, torch.full((), -math.inf, device="cuda"))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    o = (e / z) @ dense(s["v_pool"], s["v_scale"])
    s["out"].copy_(o.view(nr, H, T, G, d).permute(0, 2, 1, 3, 4).reshape(nr, T, H * G, d))
    s["lse"].copy_((m + torch.log(z)).view(nr, H, T, G).permute(0, 2, 1, 3).reshape(nr, T, H * G))
    return dict(out=s["out"], lse=s["lse"], scores=s["scores"])


def _plain_draft(s):
    c, pt = s["case"], s["page_table"].long()
    H, d, G, nr = c["hkv"], c["d"], c["hq"] // c["hkv"], c["nr"]
    L, n, step = s["seq_lens"].long().view(nr, 1, 1), s["sel_count"].long().view(nr, H, 1), s["step"].long().view(nr, 1, 1)
    a = torch.arange(s["sel_idx"].shape[-1] + 8, device="cuda").view(1, 1, -1).expand(nr, H, -1)
    sel = torch.cat([s["sel_idx"].long(), torch.zeros((nr, H, 8), dtype=torch.long, device="cuda")], dim=2)
    seen = a < n + step + 1
    pos = torch.where(seen, torch.where(a < n, sel, L + a - n), torch.zeros((), dtype=torch.long, device="cuda"))
    page = torch.gather(pt.unsqueeze(1).expand(nr, H, -1), 2, pos // PAGE).clamp_min(0)
    head = torch.arange(H, device="cuda").view(1, H, 1)
    q = s["q"].float().view(nr, H, G, d)
    x = q @ _rows(s["k_pool"], s["k_scale"], page, head, pos % PAGE).transpose(2, 3) * (1.0 / math.sqrt(d))
    x = torch.where(seen.unsqueeze(2), x, torch.full((), -math.inf, device="cuda"))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    v = _rows(s["v_pool"], s["v_scale"], page, head, pos % PAGE)
    s["out"].copy_(((e / z) @ v).view(nr, H * G, d))
    s["lse"].copy_((m + torch.log(z)).view(nr, H * G))
    return dict(out=s["out"], lse=s["lse"])


def _power_scale(amax):
    """The smallest power of two 2^e (e >= -126) with amax <= 448 * 2^e; 1 where amax is zero."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp_min(-126)
    return torch.where(amax > 0, ((e + 127) << 23).view(torch.float32), torch.ones_like(amax))   # 2^e, exactly


def _plain_append(s):
    c, T, pt = s["case"], s["T"], s["page_table"].long()
    nr = c["nr"]
    L, n = s["seq_lens"].long().view(nr, 1, 1), s["n_new"].long().view(nr, 1, 1)
    m = torch.arange(-(-T // PAGE) + 1, device="cuda").view(1, -1, 1)
    pos = (L // PAGE + m) * PAGE + torch.arange(PAGE, device="cuda").view(1, 1, PAGE)          # [nr][pages][16]
    new, old = (pos >= L) & (pos < L + n), pos < L
    there = new.any(-1)                                                                        # pages with a new row
    page = torch.gather(pt, 1, (L // PAGE + m)[:, :, 0].clamp_max(pt.shape[1] - 1)).clamp_min(0)
    row = (pos - L).clamp(0, T - 1)
    r = torch.arange(nr, device="cuda").view(nr, 1, 1)
    at, live = page[there], there.unsqueeze(-1)
    for new_rows, pool, scale in ((s["k_new"], s["k_pool"], s["k_scale"]), (s["v_new"], s["v_pool"], s["v_scale"])):
        x = new_rows[r, row][there].float().transpose(1, 2)                                    # [n][H][16][d]
        was = pool.view(torch.uint8)[at].view(F8).float() * scale[at][..., None, None]
        isnew, isold = new[there][:, None, :, None], (old & live)[there][:, None, :, None]
        x = torch.where(isnew, x, torch.where(isold, was, torch.zeros((), device="cuda")))
        sc = _power_scale(x.abs().amax((2, 3)))
        code = (x / sc[..., None, None]).to(F8).view(torch.uint8)
        keep = pool.view(torch.uint8)[at]
        pool.view(torch.uint8)[at] = torch.where(isnew | isold, code, keep)
        scale[at] = sc
    return dict(k=s["k_pool"], v=s["v_pool"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _plain_alloc(s):
    pt, T = s["page_table"], s["T"]
    nr, cols = pt.shape
    L, n, held = s["seq_lens"].long(), s["n_new"].long(), s["held"].long()
    have = s["free_count"].long()
    add = (-(-(L + n) // PAGE) - held).clamp_min(0)
    upto = add.cumsum(0)
    ok = (add == 0) | (upto <= have)
    got = torch.where(ok, add, torch.zeros_like(add))
    i = torch.arange(cols, device="cuda").view(1, cols)
    mine = (i >= held.view(nr, 1)) & (i < (held + got).view(nr, 1))
    at = (have - 1 - ((upto - add).view(nr, 1) + i - held.view(nr, 1))).clamp(0, s["free_pages"].numel() - 1)
    pt.copy_(torch.where(mine, s["free_pages"][at], pt))
    s["held_out"].copy_(held + got)
    s["free_count_out"].copy_(have - got.sum())
    s["granted"].copy_(ok)
    t = torch.arange(T, device="cuda").view(1, T)
    pos = (L.view(nr, 1) + t)
    slot = torch.gather(pt.long(), 1, (pos // PAGE).clamp_max(cols - 1)) * PAGE + pos % PAGE
    s["slots"].copy_(torch.where((t < n.view(nr, 1)) & ok.view(nr, 1), slot, torch.full_like(slot, -1)))
    return dict(table=pt, held=s["held_out"], count=s["free_count_out"], granted=s["granted"], slots=s["slots"])


def _plain_release(s):
    pt = s["page_table"]
    nr, cols = pt.shape
    held, keep = s["held"].long(), -(-s["keep_len"].long() // PAGE)
    gone = (held - keep).clamp_min(0)
    before = gone.cumsum(0) - gone
    i = torch.arange(cols, device="cuda").view(1, cols)
    out = (i >= keep.view(nr, 1)) & (i < held.view(nr, 1))
    at = s["free_count"].long() + before.view(nr, 1) + i - keep.view(nr, 1)
    s["free_pages"][at[out]] = pt[out]
    s["held_out"].copy_(held - gone)
    s["free_count_out"].copy_(s["free_count"].long() + gone.sum())
    return dict(free=s["free_pages"], held=s["held_out"], count=s["free_count_out"])


# --------------------------------------------------------------------------------- 64 bits
def _pages64(pool, scale, pages):
    """[n pages * 16][H][d] values of a list of pages."""
    x = pool[pages].to(torch.float64) * scale[pages].to(torch.float64)[:, :, None, None]
    return x.permute(0, 2, 1, 3).reshape(-1, pool.shape[1], pool.shape[3])


def _softmax64(q, k, v):
    """Rows q [H][R][d] over k, v [n][H][d]: outputs [H][R][d], log sums [H][R], logits [H][R][n]."""
    x = torch.einsum("hrd,nhd->hrn", q, k) / math.sqrt(q.shape[-1])
    z = torch.logsumexp(x, -1)
    return torch.einsum("hrn,nhd->hrd", torch.exp(x - z[..., None]), v), z, x


def exact(case, seed):
    if case["op"] in ("alloc", "release"):
        return None
    s = prepare(case, seed)
    nr, H, d = case["nr"], case["hkv"], case["d"]
    lens = _lengths(case)
    pt = s["page_table"].long()
    if case["op"] == "verify":
        T, G = case["k"] + 1, case["hq"] // H
        out, lse = torch.zeros((nr, T, H * G, d), dtype=torch.float64, device="cuda"), torch.zeros((nr, T, H * G), dtype=torch.float64, device="cuda")
        sc = None if s["scores"] is None else torch.zeros(s["scores"].shape, dtype=torch.float64, device="cuda")
        for r in range(nr):
            L = int(lens[r])
            n = L + T
            pages = pt[r, : -(-n // PAGE)]
            k, v = _pages64(s["k_pool"], s["k_scale"], pages)[:n], _pages64(s["v_pool"], s["v_scale"], pages)[:n]
            for t in range(T):
                o, z, x = _softmax64(s["q"][r, t].double().view(H, G, d), k[: L + t + 1], v[: L + t + 1])
                out[r, t], lse[r, t] = o.reshape(H * G, d), z.reshape(-1)
                if sc is not None:
                    sc[r, :, t * G:(t + 1) * G, :L] = x[:, :, :L]
        return dict(out=out, lse=lse, scores=sc)
    if case["op"] == "draft":
        G = case["hq"] // H
        out, lse = torch.zeros((nr, H * G, d), dtype=torch.float64, device="cuda"), torch.zeros((nr, H * G), dtype=torch.float64, device="cuda")
        steps = _steps(case)
        for r in range(nr):
            L, n = int(lens[r]), int(s["sel_count"][r, 0])
            block = torch.arange(L, L + int(steps[r]) + 1, device="cuda").expand(H, -1)
            pos = torch.cat([s["sel_idx"][r, :, :n].long(), block], dim=1).T                   # [n][H]
            page, head = pt[r][pos // PAGE], torch.arange(H, device="cuda").expand(pos.shape)
            k, v = ((p.view(torch.uint8)[page, head, pos % PAGE].view(F8).double() * sc[page, head].double()[..., None])
                    for p, sc in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])))
            o, z, _ = _softmax64(s["q"][r].double().view(H, G, d), k, v)
            out[r], lse[r] = o.reshape(H * G, d), z.reshape(-1)
        return dict(out=out, lse=lse)
    # append: the values over their page's scale, before any rounding
    n_new = _new_counts(case)
    res = {}
    for name, rows in (("k", s["k_new"]), ("v", s["v_new"])):
        pool, scale = s[name + "_pool"].double(), s[name + "_scale"].double()
        for r in range(nr):
            L, n = int(lens[r]), int(n_new[r])
            first, last = L // PAGE, (L + n - 1) // PAGE
            pages = pt[r, first:last + 1]
            x = _pages64(s[name + "_pool"], s[name + "_scale"], pages)                         # [pages * 16][H][d]
            a, b = L - first * PAGE, L - first * PAGE + n
            x[a:b] = rows[r, :n].double()
            top = x.clone()
            top[b:] = 0
            top = top.view(-1, PAGE, H, d).abs().amax((1, 3))
            sc = torch.full_like(top, 2.0 ** -126)
            while bool((top > F8_MAX * sc).any()):
                sc = torch.where(top > F8_MAX * sc, 2.0 * sc, sc)
            sc = torch.where(top > 0, sc, torch.ones_like(sc))
            y = (x.view(-1, PAGE, H, d) / sc[:, None, :, None]).permute(0, 2, 1, 3)            # [pages][H][16][d]
            live = (torch.arange(y.shape[0] * PAGE, device="cuda") < b).view(-1, 1, PAGE, 1)
            pool[pages] = torch.where(live, y, pool[pages])
            scale[pages] = sc
        res[name], res[name + "_scale"] = pool, scale
    return res
