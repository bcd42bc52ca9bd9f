// Rows enter the 8-bit cache.
//
// What it computes, for every page that receives a row, per KV head and for K and V apart: with
// the live rows x (the rows kept from before, at their old scale, and the new ones), the scale is
// s = 2^e, e the least integer (>= -126) with max |x| <= 448 * 2^e (s = 1 if all are zero), and
// the codes are e4m3(x / s), round to nearest even. A power of two costs e4m3 at most one of its
// 18 binades and makes both the division and a later change of scale exact (kept codes only move
// their exponent, but for those that leave the normal range); a kept page's scale that is not a
// power of two (written by someone else) is re-rounded once.
//
// Bound: HBM for prompts (2 bytes read and 1 written per element), latency for a round's rows.
// One warp per (page, KV head) of K or V: the page's 16 rows are in flight at once (eight 16-byte
// loads per lane at d = 128), the maximum is one warp reduction, and each row's codes leave as one
// 128-byte line; the eight warps of a CTA take consecutive heads, which lie side by side in the
// source rows. A page of new rows that are all finite has a short form of its own: 16 ragged prompts of
// up to 8k rows of 8 heads of 128 take 36 us a call in a row with it, 41 by itself, and took 51 us
// without; K and V in the same warp give 37 us there, but 12 us instead of 7.4 us for the 7 rows of a
// round of 32 requests. What bounds ragged prompts is the grid, pages of T rows x requests, of which
// 85% here find no rows: the same rows in 16 equal prompts take 27 us by themselves (70% of the copy
// rate), 16 prompts of 8191 rows 131 us (94%).
#include "kernels.h"
#include "kv8.cuh"

namespace s3r {

constexpr int kAppendWarps = 8;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A bf16 as a float, NaN and infinities as 0 (and `bad` raised).
__device__ __forceinline__ float finite_bf16(uint32_t bits16, bool& bad) {
  if ((bits16 & 0x7f80u) == 0x7f80u) {
    bad = true;
    return 0.f;
  }
  return __uint_as_float(bits16 << 16);
}

template <int D>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kv8_kernel(const AppendKv8Params p) {
  pdl_wait();
  constexpr int LR = D / 8;         // lanes per row (8 elements each)
  constexpr int RI = 32 / LR;       // rows per load instruction
  constexpr int NI = kPage / RI;    // load instructions per page
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int task = blockIdx.z * kAppendWarps + warp;      // K heads, then V heads
  const bool is_v = task >= p.Hkv;
  const int h = is_v ? task - p.Hkv : task;
  const int bl = blockIdx.y, m = blockIdx.x;
  const int r = p.req_ids ? p.req_ids[bl] : bl;
  const bool teller = m == 0 && task == 0 && lane == 0;   // reports for the request
  if (r < 0 || r >= p.num_requests) {
    if (teller) no_request(r, p.err);
    return;
  }
  const int L = p.seq_lens[r];
  const int f = p.first ? p.first[r] : 0;
  const int n = p.n_new ? p.n_new[r] : p.T;
  if (L < 0 || f < 0 || n < 0 || n > p.T || (int64_t)L + f + n > p.cap) {
    if (teller) set_error(p.err, S3R_ERR_DEVICE_BOUNDS);
    return;
  }
  const int start = L + f, end = start + n;
  const int pg = start / kPage + m;
  // (without rows the request's last page, which may be half full, receives none either)
  if (n == 0 || pg * kPage >= end || h >= p.Hkv) return;
  const int page = p.page_table[(size_t)r * p.max_pages + pg];
  const int row0 = lane / LR, c8 = lane % LR;
  const bool any_old = pg * kPage < start;
  // new rows: 8 bf16; kept rows: 8 codes in .x, .y. The new ones need no page and start at once.
  uint4 raw[NI];
  const __nv_bfloat16* src = (is_v ? p.v_new : p.k_new) + (size_t)r * p.kv_stride + (size_t)h * D;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int pos = pg * kPage + i * RI + row0;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (pos >= start && pos < end)
      raw[i] = __ldg(reinterpret_cast<const uint4*>(src + (size_t)(pos - start) * p.Hkv * D) + c8);
  }
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) set_error(p.err, S3R_ERR_DEVICE_BOUNDS);
    return;
  }
  uint8_t* pool = (is_v ? p.v_pool : p.k_pool) + ((size_t)page * p.Hkv + h) * (kPage * D);
  float* scale = (is_v ? p.v_scale : p.k_scale) + (size_t)page * p.Hkv + h;
  float s_old = 0.f;
  if (any_old) {
    s_old = *scale;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (pg * kPage + i * RI + row0 < start) {
        const uint2 x = *reinterpret_cast<const uint2*>(pool + (i * RI + row0) * D + c8 * 8);
        raw[i].x = x.x;
        raw[i].y = x.y;
      }
    }
  }
  // The common page, all rows new and finite: the maximum by the bits of bf16 pairs, and four
  // instructions per element in all; the general form below takes about three times that.
  uint32_t top2 = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint4 x = raw[i];
    top2 = max_u16x2(top2, max_u16x2(max_u16x2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                             max_u16x2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
  }
  const uint32_t top = __reduce_max_sync(kFull, max(top2 & 0xffffu, top2 >> 16));
  if (!any_old && top < 0x7f80u) {
    // top = 1.f * 2^x <= 1.75 * 2^(e + 8)
    int e = max((int)(top >> 7) - 127 - ((top & 0x7fu) <= 0x60u ? 8 : 7), -126);
    if (top == 0) e = 0;
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int pos = pg * kPage + i * RI + row0;
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = mul2(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u)), inv2);
        q[j] = pack_e4m3(v.x, v.y);
      }
      if (pos < end)
        *reinterpret_cast<uint2*>(pool + (i * RI + row0) * D + c8 * 8) =
            make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
    }
    if (lane == 0) *scale = __uint_as_float((uint32_t)(e + 127) << 23);
    return;
  }
  const float so = any_old ? good_scale(s_old, p.err) : 0.f;
  bool bad = false;
  // the 8 values of load i as floats
  auto values = [&](int i, float (&v)[8]) {
    const int pos = pg * kPage + i * RI + row0;
    const uint4 x = raw[i];
    if (pos >= start) {
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = finite_bf16(w[j] & 0xffffu, bad);
        v[2 * j + 1] = finite_bf16(w[j] >> 16, bad);
      }
    } else {
      const uint32_t w[4] = {x.x & 0xffffu, x.x >> 16, x.y & 0xffffu, x.y >> 16};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y = unpack_e4m3(w[j]);
        v[2 * j] = y.x * so;
        v[2 * j + 1] = y.y * so;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (!(fabsf(v[2 * j + q]) < INFINITY)) {
            bad = true;
            v[2 * j + q] = 0.f;
          }
      }
    }
  };
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    float v[8];
    values(i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
  }
  amax = warp_max(amax);
  if (bad) set_error(p.err, S3R_ERR_NONFINITE);
  // amax = 1.f * 2^x <= 1.75 * 2^(e + 8)
  const uint32_t ab = __float_as_uint(amax);
  int e = (int)(ab >> 23) - 127 - ((ab & 0x7fffffu) <= 0x600000u ? 8 : 7);
  e = max(e, -126);
  if (amax == 0.f) e = 0;
  const float s = __uint_as_float((uint32_t)(e + 127) << 23), inv = __uint_as_float((uint32_t)(127 - e) << 23);
  const bool same = any_old && s == so && !__any_sync(kFull, bad);   // kept codes stay as they are
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int pos = pg * kPage + i * RI + row0;
    if (pos >= end || (pos < start && same)) continue;
    float v[8];
    values(i, v);
    uint2 x;
    x.x = pack_e4m3(v[0] * inv, v[1] * inv) | (pack_e4m3(v[2] * inv, v[3] * inv) << 16);
    x.y = pack_e4m3(v[4] * inv, v[5] * inv) | (pack_e4m3(v[6] * inv, v[7] * inv) << 16);
    *reinterpret_cast<uint2*>(pool + (i * RI + row0) * D + c8 * 8) = x;
  }
  if (lane == 0) *scale = s;
}

int launch_append_kv8(const AppendKv8Params& p, int D, int batch, cudaStream_t stream) {
  // pages a request's T rows can touch at any offset in a page
  dim3 grid((p.T + kPage - 2) / kPage + 1, batch, (2 * p.Hkv + kAppendWarps - 1) / kAppendWarps);
  if (D == 128) launch_pdl(append_kv8_kernel<128>, grid, 32 * kAppendWarps, 0, stream, p);
  else launch_pdl(append_kv8_kernel<64>, grid, 32 * kAppendWarps, 0, stream, p);
  return cuda_status(cudaGetLastError(), "s3r_kv8_append");
}

}  // namespace s3r
