// Sparse self-draft attention over the 8-bit cache (e4m3 codes, one scale per (page, KV head)
// for K and for V), head_dim 64 and 128.
//
// What it computes: draft step i of request r lets the G query rows of each KV head attend
// A_i = S and {L, .., L+i} (S the selected positions), k_j = K[j] ks[page(j)], v_j likewise,
// as draft.cu does over the bf16 cache; the token's own row is in the cache already.
//
// Bound: HBM / L2 gather bandwidth (2 d bytes per position and KV head), latency for few rows.
// A row is one 128-byte line (d = 128), so nothing is staged: every code goes from global memory
// straight into the registers of the thread whose tensor-core fragment holds it. The order of d
// (and of the positions) within an mma.m16n8k16 is free as long as both operands agree, so a
// thread loads 16 consecutive codes of a row and feeds them to successive products:
//   S^T (16 positions x 8 rows) = K . Q^T: lane (g, t) = (lane / 4, lane % 4) loads bytes
//     [16 t, 16 t + 16) of each 64-byte half of the rows of positions g and g + 8;
//   O^T (16 d x 8 rows) += V^T . P^T: it loads d [g d/8, (g + 1) d/8) of positions 2t, 2t+1,
//     2t+8, 2t+9, pairs the codes of two positions with byte permutes and converts the pairs.
// e4m3 -> f16 is exact; q goes to f16 scaled by a power of two per row (a bf16 has 8 significant
// bits, a half 11: exact down to 2^-21 of the row's largest element, 2^-31 of it off below); P
// to f16 as 2^(z - mz + 10), z = x + log2 vs and mz its running maximum (within 2^-11, whatever
// the page scales are), the row sums from 2^(x - m) with the running maximum m of x, in fp32; ks
// multiplies the logits in fp32.
//
// Work: grid (KV head, request, chunk of A_i), 4 warps; warp w takes the chunk's batches of 32
// positions w, w + 4, .. and runs by itself (lane l resolves position l: index -> page -> row,
// scales) with an online softmax. Its K registers take the next batch's rows as soon as S is
// computed, its V registers as soon as O is, the indices run two batches ahead and the pages one,
// so that 4 to 8 KB per warp are in flight all the time (12 warps per SM). Warps merge in shared
// memory, chunks through the workspace in the last CTA of the (request, KV head). The chunk length
// follows from the launch: as many CTAs as the SMs hold at once where there is enough to read, at
// least one batch per warp.
// Measured: 32 requests of 8k to 24k, 8 KV heads, d = 128: 22 us at 5% of the cache (2.5 TB/s; the
// bf16 draft takes 31), 77 us at 20% of 24k each (4.2 TB/s, 65% of the copy rate); 26 and 95 us
// before the registers were refilled early. Chunks of up to 512 or 2048, twice the CTAs and loads
// past L1 are not faster. What bounds the 5%: each warp's chain index -> page -> row and scale ->
// product, once per 32 positions with one batch of rows in registers, and the split: the chunk follows
// from the longest set (sel_stride), not the sets' sum, so the longest of the 400 CTAs has 768
// positions where an even share of the 444 resident ones is 467.
#include "attention.cuh"
#include "draft_merge.cuh"
#include "kernels.h"
#include "kv8.cuh"

namespace s3r {

constexpr int kDraftKv8Min = 128;    // one batch of 32 positions per warp
constexpr int kDraftKv8Max = 1024;
constexpr int kDraftKv8PerSm = 3;    // resident CTAs
constexpr float kNoMax = -1e30f;     // a running maximum before its first value

// D = A (16x16 f16, row) * B (16x8 f16, col) + D, fp32 accumulation.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(128, kDraftKv8PerSm) draft_kv8_kernel(const DraftKv8Params p) {
  pdl_wait();
  constexpr int RW = 8, KC = D / 64, VW = D / 32;   // 16-byte pieces of a K row per thread; words of a V row
  constexpr int MT = D / 16;                        // m-tiles of O^T
  __shared__ float redO[4 * RW * (D + 4)];
  __shared__ float redM[4 * RW], redL[4 * RW], fw[4 * RW], Mrow[RW], Lrow[RW];
  __shared__ int s_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int kvh = blockIdx.x, bl = blockIdx.y, c = blockIdx.z;
  const int r = p.req_ids ? p.req_ids[bl] : bl;
  if (r < 0 || r >= p.num_requests) {
    if (c == 0 && kvh == 0 && tid == 0) no_request(r, p.err);
    return;
  }
  const int Hkv = p.Hkv, G = p.G;
  const int start = c * p.chunk;
  // the first batch's selected index, before the set size is known (one round trip with it)
  const int* sel = p.sel_idx + ((size_t)r * Hkv + kvh) * p.sel_stride;
  int a = start + warp * 32 + lane;      // this lane's place in A_i
  int sidx = a < p.sel_stride ? __ldg(sel + a) : -1;
  const int L = p.seq_lens[r];
  const int step = p.draft_step[r];
  const int n = p.sel_count[(size_t)r * Hkv + kvh];
  if (L < 0 || step < 0 || step >= S3R_MAX_K || (int64_t)L + step >= p.cap || n < 0 || n > p.sel_stride) {
    if (c == 0 && tid == 0) set_error(p.err, S3R_ERR_DEVICE_BOUNDS);
    return;
  }
  const int A = n + step + 1;
  const int nch = (A + p.chunk - 1) / p.chunk;
  if (c >= nch) return;
  const int end = min(A, start + p.chunk);
  const int* ptab = p.page_table + (size_t)r * p.max_pages;

  // place a of A_i -> page id (-1: nothing there; -2: out of range) and slot
  auto resolve = [&](int place, int index, int& page, int& slot) {
    page = -1;
    slot = 0;
    if (place >= end) return;
    const int pos = place < n ? index : L + (place - n);
    if (place < n && (pos < 0 || pos >= L)) {
      page = -2;
      return;
    }
    page = __ldg(ptab + (pos >> 4));
    if (page < 0 || page >= p.num_pages) page = -2;
    slot = pos & 15;
  };
  int page, slot;
  resolve(a, sidx, page, slot);

  // query rows as f16 B fragments, each row scaled by its own power of two
  uint32_t qf[4 * KC][2];
  float rf;   // of row g
  {
    uint4 w[KC][2];
    uint32_t amax = 0;
#pragma unroll
    for (int h = 0; h < KC; ++h) {
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (size_t)r * p.q_stride + (size_t)(kvh * G + g) * D + 64 * h + 16 * t);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[h][i] = g < G ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        const uint4 x = w[h][i];
        const uint32_t mx = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                     __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
        amax = max(amax, max(mx & 0xffffu, mx >> 16));
      }
    }
    amax = max(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = max(amax, __shfl_xor_sync(kFull, amax, 2));
    const int e = max((int)(amax >> 7) - 127 - 7, -120);   // largest element to [128, 256)
    const bool bad = amax >= 0x7f80u;                      // NaN or infinity: the row becomes NaN
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    rf = __uint_as_float((uint32_t)(127 + e) << 23) * p.scale * kLog2e;
    if (bad && t == 0 && c == 0 && warp == 0) set_error(p.err, S3R_ERR_NONFINITE);
#pragma unroll
    for (int h = 0; h < KC; ++h)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint4 x = w[h][s >> 1];
        const uint32_t w0 = (s & 1) ? x.z : x.x, w1 = (s & 1) ? x.w : x.y;
        auto half2_of = [&](uint32_t v) -> uint32_t {
          return bad ? 0x7fff7fffu
                     : pack_h2(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xffff0000u) * inv);
        };
        qf[4 * h + s][0] = half2_of(w0);
        qf[4 * h + s][1] = half2_of(w1);
      }
  }
  // factors of the two rows this thread holds in S^T and O^T
  const float rf0 = __shfl_sync(kFull, rf, 8 * t), rf1 = __shfl_sync(kFull, rf, 8 * t + 4);

  float o[MT][4];
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
  // running maxima of x and of z, sums relative to the former, O to the latter (- 10)
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, z0 = kNoMax, z1 = kNoMax;

  uint4 kr[4][KC];       // rows of positions g, g + 8, g + 16, g + 24
  uint32_t vr[8][VW];    // positions 2t, 2t+1, 2t+8, 2t+9 (+16)
  float ks = 0.f, vs = 0.f, ksn = 0.f, vsn = 0.f;   // this lane's position's scales: the batch's, the next one's
  // a position's row in the pools (d-byte rows); -1 for none (or a bad one): reads as zeros
  auto row_of = [&](int page, int slot) -> int {
    if (page == -2) set_error(p.err, S3R_ERR_DEVICE_BOUNDS);
    return page >= 0 ? (page * Hkv + kvh) * kPage + slot : -1;   // < 2^31 (checked at the call)
  };
  auto load_k = [&](int row) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rw = __shfl_sync(kFull, row, g + 8 * i);
#pragma unroll
      for (int h = 0; h < KC; ++h)
        kr[i][h] = rw >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.k_pool + (size_t)rw * D + 64 * h + 16 * t))
                           : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_v = [&](int row) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pp = 16 * (i >> 2) + 8 * ((i >> 1) & 1) + 2 * t + (i & 1);
      const int rw = __shfl_sync(kFull, row, pp);
      const uint8_t* src = p.v_pool + (size_t)(rw < 0 ? 0 : rw) * D + g * (D / 8);
      if constexpr (D == 128) {
        const uint4 x = rw >= 0 ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
        vr[i][0] = x.x; vr[i][1] = x.y; vr[i][2] = x.z; vr[i][3] = x.w;
      } else {
        const uint2 x = rw >= 0 ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
        vr[i][0] = x.x; vr[i][1] = x.y;
      }
    }
  };
  auto load_scales = [&](int page, float& k, float& v) {
    k = v = 0.f;
    if (page >= 0) {
      k = __ldg(p.k_scale + (size_t)page * Hkv + kvh);
      v = __ldg(p.v_scale + (size_t)page * Hkv + kvh);
    }
  };
  auto next_index = [&]() {   // the place a batch on, and its selected index
    a += 128;
    sidx = a < n ? __ldg(sel + a) : -1;
  };
  // first batch: its rows; the second's page
  int row = row_of(page, slot);
  load_scales(page, ks, vs);
  load_k(row);
  load_v(row);
  next_index();
  resolve(a, sidx, page, slot);

  for (int b = start + warp * 32; b < end; b += 128) {
    const int left = end - b;   // positions of this batch that count
    float s[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[u][i] = 0.f;
#pragma unroll
      for (int h = 0; h < KC; ++h) {
        const uint32_t x[4] = {kr[2 * u][h].x, kr[2 * u][h].y, kr[2 * u][h].z, kr[2 * u][h].w};
        const uint32_t y[4] = {kr[2 * u + 1][h].x, kr[2 * u + 1][h].y, kr[2 * u + 1][h].z, kr[2 * u + 1][h].w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mma_f16(s[u], e4m3_lo_h2(x[q]), e4m3_lo_h2(y[q]), e4m3_hi_h2(x[q]), e4m3_hi_h2(y[q]),
                  qf[4 * h + q][0], qf[4 * h + q][1]);
      }
    }
    // K's registers are free: the next batch's rows, while this one's weights are formed
    row = row_of(page, slot);
    load_scales(page, ksn, vsn);
    load_k(row);
    next_index();
    ks = good_scale(ks, p.err);
    const float lv = log2f(good_scale(vs, p.err));   // -inf: nothing of this position in O
    // logits in log2 units; positions g, g + 8 (s[0]), g + 16, g + 24 (s[1]), rows 2t, 2t + 1
    float mx0 = -INFINITY, mx1 = -INFINITY, mz0 = z0, mz1 = z1, lvp[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int pp = 16 * u + 8 * i + g;
        const float kf = __shfl_sync(kFull, ks, pp);
        lvp[u][i] = __shfl_sync(kFull, lv, pp);
        const bool in = pp < left;
        s[u][2 * i] = in ? s[u][2 * i] * kf * rf0 : -INFINITY;
        s[u][2 * i + 1] = in ? s[u][2 * i + 1] * kf * rf1 : -INFINITY;
        mx0 = fmaxf(mx0, s[u][2 * i]);
        mx1 = fmaxf(mx1, s[u][2 * i + 1]);
        mz0 = fmaxf(mz0, s[u][2 * i] + lvp[u][i]);
        mz1 = fmaxf(mz1, s[u][2 * i + 1] + lvp[u][i]);
      }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, x));
      mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, x));
      mz0 = fmaxf(mz0, __shfl_xor_sync(kFull, mz0, x));
      mz1 = fmaxf(mz1, __shfl_xor_sync(kFull, mz1, x));
    }
    const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
    // m is -inf only before any position counted (or in a NaN row): nothing to rescale then
    l0 *= m0 == -INFINITY ? 0.f : ex2(m0 - n0);
    l1 *= m1 == -INFINITY ? 0.f : ex2(m1 - n1);
    const float o0 = ex2(z0 - mz0), o1 = ex2(z1 - mz1);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      o[j][0] *= o0;
      o[j][1] *= o1;
      o[j][2] *= o0;
      o[j][3] *= o1;
    }
    m0 = n0;
    m1 = n1;
    z0 = mz0;
    z1 = mz1;
    uint32_t pf[2][2];   // P^T fragments
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // masked places give 2^-inf = 0; a row whose maximum is -inf holds NaN (2^NaN)
        const float x0 = s[u][2 * i], x1 = s[u][2 * i + 1];
        l0 += ex2(x0 - m0);
        l1 += ex2(x1 - m1);
        pf[u][i] = movm_t(pack_h2(ex2(x0 + lvp[u][i] - z0 + 10.f), ex2(x1 + lvp[u][i] - z1 + 10.f)));
      }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int wd = 0; wd < VW; ++wd) {
        // codes of positions (2t, 2t+1) and (2t+8, 2t+9), two d per permute
        const uint32_t x0 = vr[4 * u][wd], x1 = vr[4 * u + 1][wd], y0 = vr[4 * u + 2][wd], y1 = vr[4 * u + 3][wd];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t xa = __byte_perm(x0, x1, q ? 0x7362 : 0x5140), ya = __byte_perm(y0, y1, q ? 0x7362 : 0x5140);
          mma_f16(o[2 * wd + q], e4m3_lo_h2(xa), e4m3_hi_h2(xa), e4m3_lo_h2(ya), e4m3_hi_h2(ya), pf[u][0], pf[u][1]);
        }
      }
    load_v(row);
    ks = ksn;
    vs = vsn;
    resolve(a, sidx, page, slot);   // the batch after the next one's page
  }

  // warp results to shared memory: O in units of the row maximum, the V factor applied
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) {
    l0 += __shfl_xor_sync(kFull, l0, x);
    l1 += __shfl_xor_sync(kFull, l1, x);
  }
  // O relative to the row maximum: 2^(mz - m - 10) (0 in a warp without positions), by its root twice:
  // the factor itself is no normal number where all V scales are below 2^-116
  const float v0 = m0 == -INFINITY && l0 == 0.f ? 0.f : ex2(0.5f * (z0 - m0 - 10.f));
  const float v1 = m1 == -INFINITY && l1 == 0.f ? 0.f : ex2(0.5f * (z1 - m1 - 10.f));
  float* ro = redO + (size_t)warp * RW * (D + 4);
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int d0 = g * (D / 8) + 2 * j;
    *reinterpret_cast<float2*>(ro + (2 * t) * (D + 4) + d0) = make_float2(o[j][0] * v0 * v0, o[j][2] * v0 * v0);
    *reinterpret_cast<float2*>(ro + (2 * t + 1) * (D + 4) + d0) = make_float2(o[j][1] * v1 * v1, o[j][3] * v1 * v1);
  }
  if (g == 0) {
    redM[warp * RW + 2 * t] = m0;
    redM[warp * RW + 2 * t + 1] = m1;
    redL[warp * RW + 2 * t] = l0;
    redL[warp * RW + 2 * t + 1] = l1;
  }
  __syncthreads();
  auto out_row = [&](int rr) { return p.out + ((size_t)r * p.Hq + kvh * G + rr) * D; };
  auto lse_row = [&](int rr) -> float* { return p.lse ? p.lse + (size_t)r * p.Hq + kvh * G + rr : nullptr; };
  slice_weights<RW>(redM, redL, G, fw, Mrow, Lrow, tid);
  if (nch == 1) {
    slices_to_output<D, RW>(redO, fw, Mrow, Lrow, G, out_row, lse_row, tid, blockDim.x);
    return;
  }
  const size_t rec_floats = (size_t)RW * (D + 2);
  float* recs = p.part + ((size_t)(p.recs_by_id ? r : bl) * Hkv + kvh) * p.nchunk_max * rec_floats;
  slices_to_record<D, RW>(redO, fw, Mrow, Lrow, G, recs + c * rec_floats, tid, blockDim.x);
  if (!last_of(p.tickets + (size_t)r * Hkv + kvh, nch, &s_flag)) return;
  if (nch <= kDraftFastMerge) {
    combine_few_records<D, RW>(recs, rec_floats, nch, G, out_row, lse_row, tid, blockDim.x);
    return;
  }
  // more records: a warp per row, their maxima and sums one per lane, their O four at a time
  constexpr int V = D / 32;
  for (int rr = warp; rr < G; rr += 4) {
    float M = -INFINITY;
    for (int q = lane; q < nch; q += 32) M = fmaxf(M, __ldcg(recs + q * rec_floats + rr));
    M = warp_max(M);
    float lsum = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int q0 = 0; q0 < nch; q0 += 32) {
      float w = 0.f, l = 0.f;
      if (q0 + lane < nch) {
        const float ms = __ldcg(recs + (q0 + lane) * rec_floats + rr);
        l = __ldcg(recs + (q0 + lane) * rec_floats + RW + rr);
        w = ms == -INFINITY ? 0.f : exp2f(ms - M);
      }
      lsum = fmaf(w, l, lsum);
      const int cnt = min(32, nch - q0);
      const float* oq = recs + q0 * rec_floats + 2 * RW + (size_t)rr * D + lane * V;
      for (int u = 0; u < cnt; u += 4) {
        float x[4][V];
#pragma unroll
        for (int i = 0; i < 4; ++i) ld_vec<V>(oq + min(u + i, cnt - 1) * rec_floats, x[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float wi = u + i < cnt ? __shfl_sync(kFull, w, (u + i) & 31) : __shfl_sync(kFull, 0.f, 0);
#pragma unroll
          for (int j = 0; j < V; ++j) acc[j] = fmaf(wi, x[i][j], acc[j]);
        }
      }
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) lsum += __shfl_xor_sync(kFull, lsum, x);
    __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(out_row(rr) + lane * V);
#pragma unroll
    for (int i = 0; i < V; i += 2) dst[i / 2] = __floats2bfloat162_rn(acc[i] / lsum, acc[i + 1] / lsum);
    float* lp = lse_row(rr);
    if (lane == 0 && lp) *lp = (M + log2f(lsum)) * kLn2;
  }
}

// Positions per CTA: the launch's (request, KV head) sets, each up to sel_stride positions, over
// as many CTAs as are resident at once, in whole batches of the four warps.
int draft_kv8_chunk(int pairs, int sel_stride, int num_sms) {
  const int64_t want = (int64_t)kDraftKv8PerSm * num_sms;
  const int64_t per = ((int64_t)pairs * sel_stride + want - 1) / want;
  const int64_t c = (per + kDraftKv8Min - 1) / kDraftKv8Min * kDraftKv8Min;
  return (int)(c < kDraftKv8Min ? kDraftKv8Min : (c > kDraftKv8Max ? kDraftKv8Max : c));
}

static int draft_kv8_chunks(int sel_stride, int chunk) {
  return (int)(((int64_t)sel_stride + S3R_MAX_K + chunk - 1) / chunk);
}

// Records of a launch over any `batch` <= num_requests requests, which stand by their places in the
// launch: pairs * chunks, at most the larger of what the longest chunk needs and two chunks more than
// a full grid per pair. A longer list has ids out of range in it; its records stand by request
// (recs_by_id), and its chunks are no shorter than those of num_requests requests.
size_t draft_kv8_bytes(int num_requests, int Hkv, int sel_stride, int D, int num_sms) {
  const size_t pairs = (size_t)num_requests * Hkv;
  const size_t full = (size_t)kDraftKv8PerSm * num_sms + 2 * pairs;
  const size_t longest = pairs * draft_kv8_chunks(sel_stride, kDraftKv8Max);
  return align_up((full > longest ? full : longest) * 8 * (D + 2) * 4, 256);
}

int launch_draft_kv8(const DraftKv8Params& p0, int D, int batch, cudaStream_t stream) {
  DraftKv8Params p = p0;
  p.nchunk_max = draft_kv8_chunks(p.sel_stride, p.chunk);
  dim3 grid(p.Hkv, batch, p.nchunk_max);
  if (grid.z > 65535) return S3R_ERR_UNSUPPORTED;
  if (D == 128) launch_pdl(draft_kv8_kernel<128>, grid, 128, 0, stream, p);
  else launch_pdl(draft_kv8_kernel<64>, grid, 128, 0, stream, p);
  return cuda_status(cudaGetLastError(), "s3r_sparse_draft_attn_kv8");
}

}  // namespace s3r
