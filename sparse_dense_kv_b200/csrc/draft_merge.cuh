// Merging of the draft kernels' partial softmaxes: the four position slices of a CTA (one per
// warp), and the chunk records of a (request, KV head).
#pragma once

#include "common.cuh"

namespace s3r {

// Merge weights of the 4 position-slice warps of each of the G rows, once per (slice, row):
// fw[s][row] = 2^(m_s - M) (0 for an empty slice), M the rows' maximum, L = sum_s fw l_s
// (in slice order). Ends with a barrier.
template <int RW>
__device__ __forceinline__ void slice_weights(const float* redM, const float* redL, int G, float* fw,
                                              float* Mrow, float* Lrow, int tid) {
  if (tid < G) {
    float M = -INFINITY;
#pragma unroll
    for (int s = 0; s < 4; ++s) M = fmaxf(M, redM[s * RW + tid]);
    float lsum = 0.f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float ms = redM[s * RW + tid];
      const float f = (ms == -INFINITY) ? 0.f : exp2f(ms - M);
      fw[s * RW + tid] = f;
      lsum += f * redL[s * RW + tid];
    }
    Mrow[tid] = M;
    Lrow[tid] = lsum;
  }
  __syncthreads();
}

// One chunk's record [m: RW][l: RW][O: RW][D] from the slices (rows below G).
template <int D, int RW>
__device__ __forceinline__ void slices_to_record(const float* redO, const float* fw, const float* Mrow,
                                                 const float* Lrow, int G, float* rec, int tid, int nthreads) {
  constexpr int DS = D + 4;
  for (int v = tid; v < G * (D / 4); v += nthreads) {
    const int row = v / (D / 4), d0 = 4 * (v - row * (D / 4));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float f = fw[s * RW + row];
      const float4 o = *reinterpret_cast<const float4*>(redO + ((size_t)s * RW + row) * DS + d0);
      acc.x += f * o.x;
      acc.y += f * o.y;
      acc.z += f * o.z;
      acc.w += f * o.w;
    }
    *reinterpret_cast<float4*>(rec + 2 * RW + (size_t)row * D + d0) = acc;
    if (d0 == 0) {
      rec[row] = Mrow[row];
      rec[RW + row] = Lrow[row];
    }
  }
}

// The G rows of a set held by one CTA: normalised outputs and LSE straight from the slices,
// with the operations (and their order) of a one-record merge followed by the combine of
// that single record.
template <int D, int RW, class OutPtr, class LsePtr>
__device__ __forceinline__ void slices_to_output(const float* redO, const float* fw, const float* Mrow,
                                                 const float* Lrow, int G, OutPtr out_row, LsePtr lse_row,
                                                 int tid, int nthreads) {
  constexpr int DS = D + 4;
  for (int v = tid; v < G * (D / 4); v += nthreads) {
    const int row = v / (D / 4), d0 = 4 * (v - row * (D / 4));
    const float M = Mrow[row], lsum = Lrow[row];
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float f = fw[s * RW + row];
      const float4 o = *reinterpret_cast<const float4*>(redO + ((size_t)s * RW + row) * DS + d0);
      acc[0] += f * o.x;
      acc[1] += f * o.y;
      acc[2] += f * o.z;
      acc[3] += f * o.w;
    }
    const float w = (M == -INFINITY) ? 0.f : exp2f(M - M) / lsum;
    float a[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = 0.f;
      a[e] += w * acc[e];
    }
    __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(out_row(row) + d0);
    o[0] = __floats2bfloat162_rn(a[0], a[1]);
    o[1] = __floats2bfloat162_rn(a[2], a[3]);
    if (d0 == 0) {
      float* lp = lse_row(row);
      if (lp) *lp = (M + log2f(lsum)) * kLn2;
    }
  }
}

// The combine of up to kDraftFastMerge chunk records, each thread for 4 consecutive d of one
// row: the records' maxima, sums and O values are all loaded before any is used (one round
// trip), then the combine's operations in its order (row maximum, sum of the weighted
// sums, weights 2^(m_c - M) / sum, weighted sum of O over the chunks).
constexpr int kDraftFastMerge = 4;
template <int D, int RW, class OutPtr, class LsePtr>
__device__ __forceinline__ void combine_few_records(const float* recs, size_t rec_floats, int nch, int G,
                                                    OutPtr out_row, LsePtr lse_row, int tid, int nthreads) {
  for (int v = tid; v < G * (D / 4); v += nthreads) {
    const int row = v / (D / 4), d4 = v - row * (D / 4);
    float mc[kDraftFastMerge], lc[kDraftFastMerge];
    float4 x[kDraftFastMerge];
#pragma unroll
    for (int c = 0; c < kDraftFastMerge; ++c) {
      if (c < nch) {
        const float* rc = recs + c * rec_floats;
        mc[c] = __ldcg(rc + row);
        lc[c] = __ldcg(rc + RW + row);
        x[c] = __ldcg(reinterpret_cast<const float4*>(rc + 2 * RW + (size_t)row * D) + d4);
      }
    }
    float M = -INFINITY;
#pragma unroll
    for (int c = 0; c < kDraftFastMerge; ++c)
      if (c < nch) M = fmaxf(M, mc[c]);
    float lsum = 0.f;
#pragma unroll
    for (int c = 0; c < kDraftFastMerge; ++c)
      if (c < nch) lsum += (mc[c] == -INFINITY) ? 0.f : exp2f(mc[c] - M) * lc[c];
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kDraftFastMerge; ++c) {
      if (c < nch) {
        const float w = (mc[c] == -INFINITY) ? 0.f : exp2f(mc[c] - M) / lsum;
        a.x += w * x[c].x;
        a.y += w * x[c].y;
        a.z += w * x[c].z;
        a.w += w * x[c].w;
      }
    }
    __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(out_row(row) + 4 * d4);
    o[0] = __floats2bfloat162_rn(a.x, a.y);
    o[1] = __floats2bfloat162_rn(a.z, a.w);
    if (d4 == 0) {
      float* lp = lse_row(row);
      if (lp) *lp = (M + log2f(lsum)) * kLn2;
    }
  }
}

}  // namespace s3r
