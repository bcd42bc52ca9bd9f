// Device helpers of the 8-bit cache's kernels: e4m3 conversions, page scales.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace s3r {

// Two floats -> two e4m3 codes (round to nearest even, saturating; NaN stays NaN), `lo` in the
// low byte.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3_h2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(h2));
  return r;
}
// Two e4m3 codes -> f16x2 (exact: every e4m3 value is a half).
__device__ __forceinline__ uint32_t e4m3_to_h2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_lo_h2(uint32_t w) { return e4m3_to_h2((uint16_t)(w & 0xffffu)); }
__device__ __forceinline__ uint32_t e4m3_hi_h2(uint32_t w) { return e4m3_to_h2((uint16_t)(w >> 16)); }
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_e4m3(uint32_t c2) {
  const uint32_t h = e4m3_to_h2((uint16_t)c2);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// A pair of values in [0, 256] -> codes h (two) of e4m3(v) and l of e4m3(32 (v - h)). The halves in
// between hold 11 bits, so h + l / 32 is within 2^-9 of v (plus 2^-15 under the normal range).
__device__ __forceinline__ void split_e4m3x2(float2 v, uint32_t& h, uint32_t& l) {
  const uint32_t x = pack_h2(v.x, v.y);
  h = pack_e4m3_h2(x);
  const uint32_t back = e4m3_to_h2((uint16_t)h);
  const __half2 d = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&back)),
                            __half2half2(__ushort_as_half((unsigned short)0x5000)));   // 32
  l = pack_e4m3_h2(*reinterpret_cast<const uint32_t*>(&d));
}

// Packed fp32 pairs (two roundings, one instruction).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return r;
}

// A page scale as read: finite and >= 0, else reported and taken as 0.
__device__ __forceinline__ float good_scale(float s, int* err) {
  if (s >= 0.f && s < INFINITY) return s;
  set_error(err, S3R_ERR_NONFINITE);
  return 0.f;
}

// V consecutive floats (V = 2, 4) written by another kernel or CTA.
template <int V>
__device__ __forceinline__ void ld_vec(const float* p, float (&x)[V]) {
  if constexpr (V == 4) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(p));
    x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
  } else {
    const float2 t = __ldcg(reinterpret_cast<const float2*>(p));
    x[0] = t.x; x[1] = t.y;
  }
}

// Span length (tiles) of the dense kv8 verify from the launch's tiles: with at least a chunk
// (`mt` tiles) per span at kSpansPerCta spans per CTA, whole chunks of that; below, 2 spans
// per CTA, at most a chunk and at least one tile.
constexpr int kSpansPerCta = 6;
__device__ __forceinline__ int span_tiles(long long tiles, int ctas, int mt) {
  const long long per = (tiles + (long long)kSpansPerCta * ctas - 1) / ((long long)kSpansPerCta * ctas);
  if (per >= mt) return (int)((per + mt - 1) / mt * mt);
  const long long few = (tiles + 2 * ctas - 1) / (2 * ctas);
  return (int)(few < 1 ? 1 : (few > mt ? mt : few));
}

}  // namespace s3r
