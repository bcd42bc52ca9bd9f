// Dense verify attention over the 8-bit cache (e4m3 codes, one scale per (page, KV head) for
// K and for V) on the 5th-generation tensor cores, head_dim 64 and 128, up to 64 rows per KV
// head (padded to NP = 16 or 32; more than 32 as two groups of half the rows).
//
// What it computes: row (t, g) of a request at committed length L attends positions 0..L+t of
//   k_j = K[j] ks[page(j)],  v_j = V[j] vs[page(j)]
//   x_j = q . k_j / sqrt(d),  out = sum_j softmax(x)_j v_j,  lse = log sum_j exp(x_j)
// with every committed logit written when asked. The block's own rows are read from the cache
// (s3r_kv8_append puts them there first).
//
// Bound: HBM, 2 d bytes of codes per position and KV head; the score capture adds 4 bytes per
// row and position. The codes are never converted: both products run as e4m3 x e4m3
// (kind::f8f6f4, fp32 accumulation) and the bf16 side of each is split in two e4m3 parts:
//   q 2^-e = qh + ql, qh = e4m3(q 2^-e), ql = e4m3(q 2^-e - qh), the row's largest element
//     scaled to [128, 256): a bf16 value has 8 significant bits and each part holds 4, so the
//     split is exact down to 2^-10 of the row's largest element and off by at most 2^-18 of it
//     below.
//   p = 2^(x - m) vs / vref, the row's reference m (log2 units) such that the largest p so far is
//     256: m = max(x + log2(vs / vref)) - 8 (vref: the largest V scale of the span's first chunk,
//     at least 2^-40), so a weight keeps its precision next to what it contributes to the output,
//     whatever the page scales are (down to 2^-88 of vref). ph = e4m3(p),
//     pl = e4m3(32 (p - ph)): within 2^-9 of p (bf16's half step is 2^-9 of the next power of
//     two), and within 2^-23 of the largest p below the normal range.
// The two parts stand side by side along N in both products (2 NP columns), so that a tile takes 8
// MMAs of M = 128, K = 32, not 12 (both parts into one S): 49 cycles each at N = 64 (measured), some
// 390 of the 2500 that a tile of 28 rows takes.
// The scales enter in fp32: ks times the logit of its position (one tensor-memory lane = one
// position = one page), vs / vref into p, vref into O. The row sums are those of 2^(x - m) in fp32;
// m need not be the row's maximum (it is within 96 of it).
//
// Organisation: one persistent CTA per SM. A work item is a span of consecutive tiles of 128
// positions of one (request, KV head, row group); more than 32 rows are two groups of half the rows,
// neighbouring items, so that the second one's K and V come from L2. Spans are claimed from a
// counter in the workspace. A span is walked in chunks of up to kMT tiles, in two passes that are two
// stages of a pipeline, each in warps of its own: the first joins the two parts of S, applies scales
// and masks, puts the logits x in tensor memory and takes the chunk's maxima; the second forms p from
// them while the first is at the next chunk. Chunks of a span are joined in registers under a running
// reference, the spans of a (request, KV head) by a second kernel. The span length follows from the
// launch's total number of tiles: about 6 spans per CTA when there is much to read, so that the claims
// balance the SMs while the span records stay a few per cent of the traffic; with little to read, 2
// spans per CTA down to single tiles, so that a few long requests use every SM.
//   warp 0      claims spans, streams K tiles (2 KB per page, one TMA box of 16 KB when the 8 pages of
//               a tile are consecutive), publishes each chunk's page scales, splits the next span's q
//               rows into the K-major operand (the first span's: warps 8-15)
//   warp 1      streams V tiles, zeroing the rows behind the context's end (0 x NaN is NaN)
//   warp 2      issues S^T tile (128 positions x 2 NP) = K . [qh, ql]^T, a ring of kNS tiles in
//               tensor memory
//   warp 3      issues O^T (128 d x 2 NP) += V^T . [ph, pl]^T, a ring of kPT tiles of P^T
//   warps 4-7   first pass, one thread per position and all rows
//   warps 8-15  second pass, two warpgroups of half the rows each (2 RP rows, the template parameter:
//               no arithmetic on padding), one thread per position
// Both passes in the same warps, one after the other, left QK idle during the second, PV during the
// first, and every pipe waiting on one chain (331 us where this takes 300: 32 requests of 8K to
// 24K tokens, 28 rows, no capture, one B200; 362 with capture; 4 rows 181, 96 % of the measured copy
// rate, where the softmax is short).
// What bounds 28 rows: the copies take 1420 cycles of a tile's 2500. Each pass takes about 1500 beside
// them, part of it waiting for instructions to be fetched (the size of the code counts, hence the
// templates and the cold parts out of line); the rest is the chunk's boundary, where the second pass
// waits for the chunk's maxima and the first for the logits' buffer. 16 rows show it: 191 us in chunks
// of 8 tiles with four S slots, 238 in the instance of 20 rows (4 tiles, two slots). From there the
// rows' arithmetic adds: 255 us at 20 rows, 290 at 24, 298 at 28. All rings hand over tile by tile.
// Every wait is bounded (S3R_ERR_TIMEOUT, as in verify_tc.cu).
#include <type_traits>

#include "kernels.h"
#include "kv8.cuh"
#include "tcgen05.cuh"

namespace s3r {
namespace kv8 {

using namespace tc;

constexpr int kPos = 128;
constexpr int kThreads = 512;
constexpr int kPWarp0 = 8, kPWarps = 8;   // second pass: 8 warps
constexpr int kTileBytes = kPos * 128;    // 16 KB: 128 positions x 128 bytes (d = 64: half zero)
constexpr int kRing = 16;
constexpr int kScaleBufs = 8;             // chunks whose page scales are held
// V scales: vs / vref is at most 2^88, since vref >= 2^-40 and larger scales than 2^48 are refused,
// and its logarithm counts as at least -88, so that the terms of a row sum lie between 2^-80 (a
// logit at the reference's) and 2^96. Between chunks and between spans the reference can rise by
// 176 with the logits where they were. What such a step leaves of O is below 2^-38 of what joins it
// (2^-126 times 2^88 of the spans' vref) and may go to zero; a row sum of 2^96 must come through
// as 2^-80, so sums are scaled by 2^(step / 2) twice.
constexpr float kMaxVScale = 0x1p48f, kMaxRatio = 88.f;
constexpr int kScaleFloats = 196;         // ks, vs / vref, log2 of that (>= -kMaxRatio) [64] each; vref; pad
constexpr int kMaxSt = 6;                 // ring stages
constexpr int kBarBytes = 1792;           // barriers, flags, the ring of spans
constexpr int kMaxBatch = 256;            // requests per launch (larger batches: several launches)
// plan area of the workspace (written by the attention kernel for the merge): span length in
// tiles, then the prefix of per-request span counts
constexpr int kPlanInts = 512;
static_assert(kMaxBatch + 2 <= kPlanInts, "plan area");

// Instruction descriptor of kind::f8f6f4: e4m3 A and B, fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// ACC: add to D. The issuing warp stays converged, its control flow and addresses warp-uniform, and
// one elected lane executes the MMAs and commits: the operands then come from uniform registers and
// an MMA leaves every 49 cycles (measured). From a diverged `if (lane == 0)` the same four MMAs and
// commit took 316 to 450 cycles alone and 800 beside the softmax warps, and the two issuers, each
// needed by one of the softmax's passes, bounded the kernel.
template <bool ACC>
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n .reg .b32 l;\n elect.sync l|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// wait_bar with its polling out of line: inlined some thirty times, the loops were most of a 170 KB
// kernel whose warps spent a third of their time waiting for instructions.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int limit) {
#pragma unroll 1
  for (int i = 0; i < limit; ++i) {
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    if ((i & 255) == 255 && __any_sync(kFull, *abort_flag != 0)) return false;
  }
  if ((threadIdx.x & 31) == 0) {
    *abort_flag = 1;
    set_error(err, S3R_ERR_TIMEOUT);
  }
  __syncwarp();
  return false;
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err,
                                          int limit) {
  if (__builtin_expect(__all_sync(kFull, mbar_try_wait(bar, parity)), 1)) return true;
  return wait_slow(bar, parity, abort_flag, err, limit);
}

// RP: pairs of rows per warpgroup (1..8).
template <int RP>
struct Cfg {
  static constexpr int NP = RP <= 4 ? 16 : 32;   // padded rows
  static constexpr int NH = NP / 2;              // columns of a warpgroup's part
  static constexpr int NR = 2 * RP;              // rows of a warpgroup
  // Tensor memory (512 columns): two O buffers of 2 NP columns, the S ring (2 NP columns per tile:
  // per half of the rows NH of qh, NH of ql), the logits of two chunks (NP columns per tile).
  static constexpr int kNS = NP == 16 ? 4 : 2;
  static constexpr int kMT = NP == 16 ? 8 : 4;   // tiles per chunk
  static constexpr int kSCol0 = 4 * NP;
  static constexpr int kXCol0 = kSCol0 + kNS * 2 * NP;
  static_assert(kXCol0 + 2 * kMT * NP <= 512 && kMT <= 8, "tensor memory budget");
  static constexpr int kPRow = 2 * NP;           // bytes of P^T per position: 32- or 64-byte swizzle
  static constexpr int kPTile = kPos * kPRow;
  static constexpr uint32_t kPSwz = NP == 16 ? 6u : 4u;
  static constexpr int kKSt = 6, kVSt = 4, kPT = 4;   // K, V and P^T ring stages
  static_assert(kKSt <= kMaxSt && kVSt == kPT && kNS <= kKSt, "shared completion barriers");
  static constexpr int kQBytes = 2 * NP * 128;   // one Q buffer: 2 NP rows of 128 bytes
  static constexpr int kKOff = 0;
  static constexpr int kVOff = kKSt * kTileBytes;
  static constexpr int kQOff = kVOff + kVSt * kTileBytes;
  static constexpr int kPOff = kQOff + 2 * kQBytes;
  static constexpr int kRedOff = kPOff + kPT * kPTile;
  // floats: redM [2][4 warps][NP]; redL [2][8 warps][NH]; references, factors [4][3][NP]; rs [8][NP];
  // scales [8][196]
  static constexpr int kRedFloats = 2 * 4 * NP + 2 * 8 * NH + 4 * 3 * NP + 8 * NP + kScaleBufs * kScaleFloats;
  static constexpr int kPrefOff = kRedOff + kRedFloats * 4;
  static constexpr int kLenOff = kPrefOff + (kMaxBatch + 4) * 4;
  static constexpr int kRidOff = kLenOff + kMaxBatch * 4;
  static constexpr int kBarOff = (kRidOff + kMaxBatch * 4 + 63) / 64 * 64;
  static constexpr int kSmem = kBarOff + kBarBytes + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kQOff % 1024 == 0 && kPOff % 1024 == 0 && kRedOff % 16 == 0, "operand alignment");
};

// A span of tiles [t0, t1) of (request r, KV head kvh), one of nsp, for the row group from g0; L
// committed positions. id < 0: the launch has no more work.
struct Span {
  int id, r, kvh, nsp, L, t0, t1, g0;
};

struct Bars {
  uint64_t kfull[kMaxSt], ktma[kMaxSt];
  uint64_t vfull[kMaxSt], vtma[kMaxSt];
  // One commit per tile and product (a commit costs the issuing thread more than an MMA): QK of the
  // tile in K stage s is complete (the stage is free, its S is there; S slots are fewer than
  // stages, so no barrier runs a phase ahead of the softmax); PV of the tile in V stage = P slot s.
  uint64_t qkd[kMaxSt], pvd[kMaxSt];
  uint64_t sempty[kMaxSt], pfull[kMaxSt];
  uint64_t q_full[2], q_empty[2];        // per span parity
  uint64_t q0;                           // the first span's q rows
  uint64_t x_full[2], x_empty[2];        // per chunk parity: its logits are in tensor memory; have been read
  uint64_t sm_done[kScaleBufs];          // chunk's second pass is over
  uint64_t sc_full[kScaleBufs];          // chunk's page scales are in shared memory
  uint64_t o_full[2], o_empty[2];        // per chunk parity
  uint64_t fin[2];
  uint64_t wg[3];                        // the second pass's two warpgroups, the first pass's
  uint64_t item_bar[kRing];
  int4 span[kRing][2];                   // the CTA's m-th span at m % kRing
  uint32_t tmem_base;
  int abort_flag;
  int span_tiles;                        // tiles per span of this launch
};
static_assert(sizeof(Bars) <= kBarBytes && sizeof(Span) == 32, "barrier block");

__device__ __forceinline__ Span make_span(int id, const int* pref, const int* lens_s, const int* rid_s,
                                          int batch, const VerifyKv8Params& p, int st) {
  int lo = 0, hi = batch;   // largest b with pref[b] <= id
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] <= id) lo = mid;
    else hi = mid;
  }
  Span x;
  x.id = id;
  const int rem = id - pref[lo];
  x.nsp = (pref[lo + 1] - pref[lo]) / (p.Hkv * p.ngroups);
  const int pair = rem / p.ngroups;
  x.g0 = (rem - pair * p.ngroups) * p.Rg;
  x.kvh = pair / x.nsp;
  x.r = rid_s[lo];
  x.L = lens_s[lo];
  x.t0 = (pair - x.kvh * x.nsp) * st;
  x.t1 = min(x.t0 + st, (x.L + p.T + kPos - 1) / kPos);
  return x;
}

// Reduce v[0..N-1] over the warp's lanes with `op`, halving the values at each exchange instead
// of reducing each one by itself (N = 28: 31 shuffles, not 140). Lane l ends up with the result
// of column col_of(l), the same one in every lane that shares it.
template <int N>
struct ColReduce {
  static constexpr int NP2 = N <= 2 ? 2 : (N <= 4 ? 4 : (N <= 8 ? 8 : (N <= 16 ? 16 : 32)));   // padded to a power of two
  // column that lane l holds after run()
  __device__ __forceinline__ static int col_of(int lane) {
    int c = 0;
#pragma unroll
    for (int w = NP2 / 2, b = 16; w >= 1; w >>= 1, b >>= 1)
      if (lane & b) c += w;
    return c;
  }
  template <class Op>
  __device__ __forceinline__ static float run(const float (&v)[N], int lane, float pad, Op op) {
    float x[NP2];
#pragma unroll
    for (int i = 0; i < NP2; ++i) x[i] = i < N ? v[i] : pad;
    int b = 16;
#pragma unroll
    for (int w = NP2 / 2; w >= 1; w >>= 1) {
      const bool up = (lane & b) != 0;
#pragma unroll
      for (int i = 0; i < w; ++i) {
        const float send = up ? x[i] : x[i + w];
        const float keep = up ? x[i + w] : x[i];
        x[i] = op(keep, __shfl_xor_sync(kFull, send, b));
      }
      b >>= 1;
    }
    for (; b >= 1; b >>= 1) x[0] = op(x[0], __shfl_xor_sync(kFull, x[0], b));
    return x[0];
  }
};

// Values of a tensor-memory load may be used from here on: ties the registers behind the wait.
template <int N>
__device__ __forceinline__ void tmem_tie(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// This warp's 32 lanes x 8 or 16 consecutive columns.
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15]))
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ready(float (&v)[N]) {
  tmem_wait_ld();
  tmem_tie(v);
}

// CAP: committed logits are written (their stores, skipped over, would still cost the other case a
// tenth of its time in instruction fetches).
template <int RP, int D, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    verify_kv8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmK8, const __grid_constant__ CUtensorMap tmV8,
                      const VerifyKv8Params p, int batch) {
  pdl_wait();
  using C = Cfg<RP>;
  constexpr int NP = C::NP, NH = C::NH, NR = C::NR;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  float* redM = reinterpret_cast<float*>(smem + C::kRedOff);   // [2][4][NP] warp maxima (chunk parity)
  float* redL = redM + 2 * 4 * NP;                              // [2][8][NH] warp sums (span parity)
  float* refs = redL + 2 * 8 * NH;                              // [4][3][NP] chunk & 3: -reference, root of the step, reference
  float* rs = refs + 4 * 3 * NP;                                // [8][NP] q row factor 2^e log2(e) / sqrt(d)
  float* scs = rs + 8 * NP;                                     // [8][196] page scales
  int* pref = reinterpret_cast<int*>(smem + C::kPrefOff);
  int* lens_s = reinterpret_cast<int*>(smem + C::kLenOff);
  int* rid_s = reinterpret_cast<int*>(smem + C::kRidOff);
  Bars* B = reinterpret_cast<Bars*>(smem + C::kBarOff);
  volatile int* abort_flag = &B->abort_flag;

  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  const int T = p.T, G = p.G, R = p.R, Hkv = p.Hkv, HG = p.Hkv * p.ngroups;
  const uint32_t sbase = smem_u32(smem);

  // ---- set-up: lengths, span length, span prefix, barriers, tensor memory
  for (int b = tid; b < batch; b += blockDim.x) {
    const int r = p.req_ids ? p.req_ids[p.req_off + b] : p.req_off + b;
    const bool known = r >= 0 && r < p.num_requests;
    const int L = known ? p.seq_lens[r] : -1;
    const bool fits = L >= 0 && L <= p.cap - T;
    if (!fits && blockIdx.x == 0) no_request(r, p.err);
    rid_s[b] = known ? r : 0;
    lens_s[b] = L;
    pref[b + 1] = fits ? (L + T + kPos - 1) / kPos : 0;   // tiles, turned into span counts below
  }
  if (tid == 0) {
    for (int s = 0; s < C::kKSt; ++s) {
      mbar_init(smem_u32(&B->kfull[s]), 1);
      mbar_init(smem_u32(&B->ktma[s]), 1);
      mbar_init(smem_u32(&B->qkd[s]), 1);
    }
    for (int s = 0; s < C::kVSt; ++s) {
      mbar_init(smem_u32(&B->vfull[s]), 1);
      mbar_init(smem_u32(&B->vtma[s]), 1);
      mbar_init(smem_u32(&B->pvd[s]), 1);
      mbar_init(smem_u32(&B->pfull[s]), 8);
    }
    for (int s = 0; s < C::kNS; ++s) mbar_init(smem_u32(&B->sempty[s]), 4);
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&B->q_full[b]), 1);
      mbar_init(smem_u32(&B->q_empty[b]), 1);
      mbar_init(smem_u32(&B->x_full[b]), 4);
      mbar_init(smem_u32(&B->x_empty[b]), 8);
      mbar_init(smem_u32(&B->o_full[b]), 1);
      mbar_init(smem_u32(&B->o_empty[b]), 8);
      mbar_init(smem_u32(&B->fin[b]), 1);
      mbar_init(smem_u32(&B->wg[b]), 4);
    }
    for (int i = 0; i < kScaleBufs; ++i) {
      mbar_init(smem_u32(&B->sc_full[i]), 1);
      mbar_init(smem_u32(&B->sm_done[i]), 8);
    }
    mbar_init(smem_u32(&B->wg[2]), 4);
    mbar_init(smem_u32(&B->q0), kPWarps);
    for (int i = 0; i < kRing; ++i) mbar_init(smem_u32(&B->item_bar[i]), 1);
    B->abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&B->tmem_base), 512);
    tmem_relinquish();
  }
  for (int i = tid; i < 2 * C::kQBytes / 16; i += kThreads)   // operand rows that no q row fills stay zero
    *reinterpret_cast<uint4*>(smem + C::kQOff + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  __syncthreads();
  if (warp == 0) {
    const int per = (batch + 31) / 32;
    const int b0 = lane * per, b1 = min(batch, b0 + per);
    long long tiles = 0;
    for (int b = b0; b < b1; ++b) tiles += pref[b + 1];
#pragma unroll
    for (int o = 16; o; o >>= 1) tiles += __shfl_xor_sync(kFull, tiles, o);
    const int st = span_tiles(tiles * HG, (int)gridDim.x, C::kMT);
    int local = 0;
    for (int b = b0; b < b1; ++b) local += HG * ((pref[b + 1] + st - 1) / st);
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    int run = incl - local;
    for (int b = b0; b < b1; ++b) {
      run += HG * ((pref[b + 1] + st - 1) / st);
      pref[b + 1] = run;
    }
    if (lane == 0) {
      pref[0] = 0;
      B->span_tiles = st;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, B->tmem_base, 0);
  const int nitems = pref[batch], st = B->span_tiles;
  if (blockIdx.x == 0)   // the merge's plan
    for (int b = tid; b <= batch + 1; b += blockDim.x) p.plan[b] = b == 0 ? st : pref[b - 1];

  // A CTA's first span is blockIdx.x, later ones come from the launch's counter; the K producer
  // claims them and publishes them in a ring (id < 0: no more work).
  auto read_span = [&](int m, Span& x) {
    const int4 a = B->span[m & (kRing - 1)][0], b = B->span[m & (kRing - 1)][1];
    x.id = a.x; x.r = a.y; x.kvh = a.z; x.nsp = a.w;
    x.L = b.x; x.t0 = b.y; x.t1 = b.z; x.g0 = b.w;
  };
  auto ring_span = [&](int m, Span& x) -> bool {   // false: no more work, or the wait gave up
    if (!wait_warp(smem_u32(&B->item_bar[m & (kRing - 1)]), (uint32_t)(m / kRing) & 1u, abort_flag, p.err, p.wait_limit))
      return false;
    read_span(m, x);
    return x.id >= 0;
  };
  auto waitb = [&](uint64_t* bar, int phase) -> bool {
    return wait_warp(smem_u32(bar), (uint32_t)phase & 1u, abort_flag, p.err, p.wait_limit);
  };

  // q rows of span m -> operand buffer m & 1: a warp takes RI rows at a time, LR lanes to a row
  // (8 elements each).
  constexpr int LR = D / 8, RI = 32 / LR;
  const int c8 = lane % LR;
  auto load_q = [&](const Span& x, int j, int rows) -> uint4 {   // row j
    if (j >= rows) return make_uint4(0, 0, 0, 0);
    const int t = (x.g0 + j) / G, gq = x.g0 + j - t * G;
    return *reinterpret_cast<const uint4*>(p.q + (((size_t)x.r * T + t) * p.Hq + x.kvh * G + gq) * D + c8 * 8);
  };
  auto split_row = [&](const uint4 raw, int j, int rows, int m) {
    // largest |q| of the row by its bits (NaN above infinity above every finite value)
    uint32_t a = __vmaxu2(__vmaxu2(raw.x & 0x7fff7fffu, raw.y & 0x7fff7fffu),
                          __vmaxu2(raw.z & 0x7fff7fffu, raw.w & 0x7fff7fffu));
    uint32_t amax = max(a & 0xffffu, a >> 16);
#pragma unroll
    for (int o = LR / 2; o; o >>= 1) amax = max(amax, __shfl_xor_sync(kFull, amax, o));
    // the largest element's exponent goes to 2^7; a row of tiny values is not scaled past 2^120
    const int e = max((int)(amax >> 7) - 127 - 7, -120);
    const bool bad = amax >= 0x7f80u;   // NaN or infinity: the row's logits become NaN
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t hh = 0, ll = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t v = w[2 * i + u];
        const float f0 = __uint_as_float(v << 16) * inv, f1 = __uint_as_float(v & 0xffff0000u) * inv;
        const uint32_t h2 = pack_e4m3(f0, f1);
        const float2 hf = unpack_e4m3(h2);
        const uint32_t l2 = pack_e4m3(f0 - hf.x, f1 - hf.y);
        hh |= h2 << (16 * u);
        ll |= l2 << (16 * u);
      }
      hi[i] = bad ? 0x7f7f7f7fu : hh;
      lo[i] = bad ? 0x7f7f7f7fu : ll;
    }
    if (j < rows) {
      const int w = j / NR, nh = w * NP + j - w * NR, nl = nh + NH;   // operand rows of the two parts
      uint8_t* dst = smem + C::kQOff + (m & 1) * C::kQBytes + (c8 & 1) * 8;
      *reinterpret_cast<uint2*>(dst + nh * 128 + (((c8 >> 1) ^ (nh & 7)) << 4)) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(dst + nl * 128 + (((c8 >> 1) ^ (nl & 7)) << 4)) = make_uint2(lo[0], lo[1]);
      if (c8 == 0) {
        rs[(m & 7) * NP + w * NH + j - w * NR] = __uint_as_float((uint32_t)(127 + e) << 23) * p.scale * kLog2e;
        if (bad) set_error(p.err, S3R_ERR_NONFINITE);
      }
    }
  };
  auto zero_factors = [&](int rows, int m) {   // of the rows behind the last one
#pragma unroll 1
    for (int j = rows + lane; j < 2 * NR; j += 32) rs[(m & 7) * NP + j / NR * NH + j % NR] = 0.f;
  };

  if (warp <= 1) {
    // ============================================================ producers ====
    const bool is_v = warp == 1;
    const CUtensorMap* map = is_v ? &tmV : &tmK;
    const CUtensorMap* map8 = is_v ? &tmV8 : &tmK8;
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
      asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map8)) : "memory");
    }
    const int nst = is_v ? C::kVSt : C::kKSt;
    const int roff = is_v ? C::kVOff : C::kKOff;
    uint64_t* full = is_v ? B->vfull : B->kfull;
    uint64_t* empty = is_v ? B->pvd : B->qkd;
    uint64_t* tmab = is_v ? B->vtma : B->ktma;
    const uint32_t sb = __shfl_sync(kFull, sbase, 0);
    float vref = 1.f;          // (K producer)
    int g = 0, slot = 0, lap = 0;   // tiles issued; the ring's position
    uint32_t tma_phase = 0;    // bit s: phase of tmab[s]
    bool stop = false;
    // Page ids of the chunk [t0, t1), two per lane (-1 past the context or outside the pool).
    auto fetch_ids = [&](const Span& x, int t0, int t1, int& a, int& b) {
      const int* ptab = p.page_table + (size_t)x.r * p.max_pages;
      const int npg = (t1 - t0) * 8, pg0 = t0 * 8, pend = (x.L + T + kPage - 1) / kPage;
      a = lane < npg && pg0 + lane < pend ? ptab[pg0 + lane] : -1;
      b = lane + 32 < npg && pg0 + lane + 32 < pend ? ptab[pg0 + lane + 32] : -1;
    };
    const bool el = elect_one();
    // The pages of a chunk: which are in the context, which of those are in the pool, which follow
    // the one before (bit i: page i of the chunk). Found once per chunk; a tile is a byte of each.
    uint64_t want = 0, good = 0, next = 0;
    auto survey = [&](const Span& x, int t0, int t1, int ida, int idb) {
      const int left = (x.L + T + kPage - 1) / kPage - t0 * 8, npg = min(left, (t1 - t0) * 8);
      auto one = [&](int id, int i, int before) -> void {
        const bool w = i < npg, g2 = w && id >= 0 && id < p.num_pages;
        const int sh = i & 32;
        want |= (uint64_t)__ballot_sync(kFull, w) << sh;
        good |= (uint64_t)__ballot_sync(kFull, g2) << sh;
        next |= (uint64_t)__ballot_sync(kFull, id == before + 1) << sh;
      };
      want = good = next = 0;
      one(ida, lane, __shfl_up_sync(kFull, ida, 1));
      if (C::kMT > 4) one(idb, lane + 32, __shfl_up_sync(kFull, idb, 1));
      if (want != good && lane == 0) set_error(p.err, S3R_ERR_DEVICE_BOUNDS);
    };
    auto load_tile = [&](const Span& x, int t, int u, int ida, int idb) {   // u: tile of the chunk
      const int s = slot;
      if (g >= nst && !waitb(&empty[s], lap - 1)) {
        stop = true;
        return;
      }
      if (++slot == nst) {   // (counted: a division by the runtime ring size costs more than the copy)
        slot = 0;
        ++lap;
      }
      const uint32_t dst = sb + roff + s * kTileBytes;
      const uint32_t okmask = (uint32_t)(good >> (8 * u)) & 0xFFu, wantmask = (uint32_t)(want >> (8 * u)) & 0xFFu;
      const bool run = okmask == 0xFFu && ((uint32_t)(next >> (8 * u)) & 0xFEu) == 0xFEu;   // 8 consecutive ids
      const int Lc = x.L + T;
      // rows that must read as zero: a bad page's, and for V every row behind the context
      const bool patch = okmask != wantmask || (is_v && (t + 1) * kPos > Lc);
      const uint32_t landing = smem_u32(patch ? &tmab[s] : &full[s]);
      const int id0 = __shfl_sync(kFull, C::kMT > 4 && u >= 4 ? idb : ida, (8 * u) & 31);
      ++g;
      if (__builtin_expect(run && !patch, 1)) {
        if (el) {
          mbar_arrive_expect_tx(landing, 8 * kPage * 128);
          tma_load_4d(dst, map8, 0, 0, x.kvh, id0, landing);
        }
        __syncwarp();
        return;
      }
      const int id = __shfl_sync(kFull, C::kMT > 4 && u >= 4 ? idb : ida, (8 * u + (lane & 7)) & 31);
      if (lane == 0) mbar_arrive_expect_tx(landing, (uint32_t)__popc(okmask) * kPage * 128);
      __syncwarp();
      if (lane < 8 && (okmask & (1u << lane))) tma_load_4d(dst + lane * kPage * 128, map, 0, 0, x.kvh, id, landing);
      if (patch) {
        if (!waitb(&tmab[s], (tma_phase >> s) & 1)) {
          mbar_wait(smem_u32(&tmab[s]), (tma_phase >> s) & 1);   // its copies land before exit
          if (lane == 0) mbar_arrive(smem_u32(&full[s]));        // (for the wait below)
          stop = true;
          return;
        }
        tma_phase ^= 1u << s;
#pragma unroll 1
        for (int idx = lane; idx < kPos * 8; idx += 32) {
          const int row = idx >> 3;
          if ((okmask & (1u << (row >> 4))) && !(is_v && t * kPos + row >= Lc)) continue;
          *reinterpret_cast<uint4*>(smem + roff + s * kTileBytes + idx * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&full[s]));
      }
      __syncwarp();
    };
    // the CTA's m-th span: claimed and published by the K producer, read by the V producer
    auto next_span = [&](int m, Span& x) -> bool {
      if (is_v) return ring_span(m, x);
      int id = (int)blockIdx.x;
      if (m > 0) {
        int v = 0;
        if (lane == 0) v = atomicAdd(p.sched, 1);
        id = __shfl_sync(kFull, v, 0) + (int)gridDim.x;
      }
      if (id < nitems) x = make_span(id, pref, lens_s, rid_s, batch, p, st);
      else x.id = -1;
      if (lane == 0) {
        const int slot = m & (kRing - 1);
        B->span[slot][0] = make_int4(x.id, x.r, x.kvh, x.nsp);
        B->span[slot][1] = make_int4(x.L, x.t0, x.t1, x.g0);
        mbar_arrive(smem_u32(&B->item_bar[slot]));   // release: the span is visible
      }
      __syncwarp();
      return x.id >= 0;
    };
    // q rows of span m (K producer, m > 0), once the QK of span m - 2 has read the buffer
    auto split_q = [&](const Span& x, int m) -> bool {
      if (m >= 2 && !waitb(&B->q_empty[m & 1], (m - 2) >> 1)) return false;
      const int rows = min(p.Rg, R - x.g0);
      constexpr int kAhead = 8;   // loads in flight
      uint4 raw[kAhead];
#pragma unroll 1
      for (int jb = 0; jb < rows; jb += kAhead * RI) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) raw[i] = load_q(x, jb + i * RI + lane / LR, rows);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (jb + i * RI >= rows) break;
          split_row(raw[i], jb + i * RI + lane / LR, rows, m);
        }
      }
      zero_factors(rows, m);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&B->q_full[m & 1]));
      return true;
    };
    // The chunk after (x, t0): the next of the span, or the first of the next span.
    int m = 0, n = 0;   // span and chunk counters
    Span x{};
    int t0 = 0, t1 = 0, ida = -1, idb = -1;
    bool more = next_span(0, x);
    if (more) {
      t0 = x.t0;
      t1 = min(t0 + C::kMT, x.t1);
      fetch_ids(x, t0, t1, ida, idb);
      // the first span's q rows are the second pass's warps' (here: the barrier's phase)
      if (!is_v && lane == 0) mbar_arrive(smem_u32(&B->q_full[0]));
    }
    // page scales of the next chunk (K producer), loaded while the current one streams
    float ka = 0.f, kb = 0.f, va = 0.f, vb = 0.f;
    auto fetch_scales = [&](const Span& y) {
      ka = kb = va = vb = 0.f;
      if (ida >= 0 && ida < p.num_pages) {
        ka = __ldg(p.k_scale + (size_t)ida * Hkv + y.kvh);
        va = __ldg(p.v_scale + (size_t)ida * Hkv + y.kvh);
      }
      if (C::kMT > 4 && idb >= 0 && idb < p.num_pages) {
        kb = __ldg(p.k_scale + (size_t)idb * Hkv + y.kvh);
        vb = __ldg(p.v_scale + (size_t)idb * Hkv + y.kvh);
      }
    };
    auto good_v_scale = [&](float v) -> float {
      v = good_scale(v, p.err);
      if (v > kMaxVScale) set_error(p.err, S3R_ERR_NONFINITE);
      return fminf(v, kMaxVScale);
    };
    if (more && !is_v) fetch_scales(x);
    while (more && !stop && !aborted(abort_flag)) {
      survey(x, t0, t1, ida, idb);
      // at most four chunks ahead of the second pass: what the scale buffers and the span ring hold
      if (!is_v && n >= 4 && !waitb(&B->sm_done[(n - 4) & (kScaleBufs - 1)], (n - 4) / kScaleBufs)) break;
      load_tile(x, t0, 0, ida, idb);
      if (stop) break;
      if (!is_v) {
        float* sc = scs + (n & (kScaleBufs - 1)) * kScaleFloats;
        va = good_v_scale(va);
        vb = good_v_scale(vb);
        // the span's unit of V scales: the largest of its first chunk, at least 2^-40
        if (t0 == x.t0) vref = fmaxf(warp_max(fmaxf(va, vb)), 0x1p-40f);
        const float inv = 1.f / vref, ra = va * inv, rb = vb * inv;
        sc[lane] = good_scale(ka, p.err);
        sc[lane + 32] = good_scale(kb, p.err);
        sc[64 + lane] = ra;
        sc[64 + lane + 32] = rb;
        sc[128 + lane] = fmaxf(log2f(ra), -kMaxRatio);
        sc[128 + lane + 32] = fmaxf(log2f(rb), -kMaxRatio);
        if (lane == 0) sc[192] = vref;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&B->sc_full[n & (kScaleBufs - 1)]));
      }
      // what comes next is claimed and its page ids are fetched while this chunk streams
      int nt0 = t1, na = -1, nb = -1;
      Span xn = x;
      if (t1 >= x.t1) {
        more = next_span(++m, xn);
        nt0 = xn.t0;
      }
      const int nt1 = min(nt0 + C::kMT, xn.t1);
      if (more) {
        fetch_ids(xn, nt0, nt1, na, nb);
        if (!is_v && t1 >= x.t1 && !split_q(xn, m)) stop = true;
      }
#pragma unroll 1
      for (int t = t0 + 1; t < t1 && !stop; ++t) load_tile(x, t, t - t0, ida, idb);
      x = xn;
      t0 = nt0;
      t1 = nt1;
      ida = na;
      idb = nb;
      if (more && !is_v) fetch_scales(x);
      ++n;
    }
    // nothing may still be landing in this ring when the CTA exits, also after an abort
    for (int q = g - nst > 0 ? g - nst : 0; q < g; ++q) mbar_wait(smem_u32(&full[q % nst]), (q / nst) & 1);
  } else if (warp <= 3) {
    // ==================================================================== MMA issuers ====
    // Warp 2: QK, warp 3: PV.
    auto uni = [](int v) -> int { return __shfl_sync(kFull, v, 0); };
    const bool el = elect_one();
    const uint32_t sb = uni((int)sbase), bars = uni((int)smem_u32(B));
    auto bar_at = [&](const uint64_t* b0, int i) -> uint32_t {
      return bars + (uint32_t)(reinterpret_cast<const uint8_t*>(b0) - reinterpret_cast<const uint8_t*>(B)) + 8 * i;
    };
    bool ok = true;
    int g = 0, n = 0;   // tiles, chunks
    if (warp == 2) {
      int s = 0, lap = 0;   // position in the K ring
      constexpr uint32_t kId = idesc_e4m3(kPos, 2 * NP, false, false);
      const uint64_t kd = sdesc(sb + C::kKOff, 16, 1024, 2), qd = sdesc(sb + C::kQOff, 16, 1024, 2);
#pragma unroll 1
      for (int m = 0; ok; ++m) {
        Span x;
        if (!ring_span(m, x) || !waitb(m == 0 ? &B->q0 : &B->q_full[m & 1], m >> 1)) break;
        const int tb = uni(x.t0), te = uni(x.t1);
        const uint64_t qm = qd + (m & 1) * (C::kQBytes >> 4);
#pragma unroll 1
        for (int t0 = tb; t0 < te && ok; t0 += C::kMT) {
          const int t1 = min(t0 + C::kMT, te);
#pragma unroll 1
          for (int t = t0; t < t1; ++t, ++g) {
            const int d = g % C::kNS;
            if (!waitb(&B->kfull[s], lap) || (g >= C::kNS && !waitb(&B->sempty[d], g / C::kNS - 1))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t km = kd + s * (kTileBytes >> 4);
            const uint32_t sd = tmem + C::kSCol0 + d * 2 * NP, done = bar_at(B->qkd, s);
            if (el) {
              mma_e4m3<false>(sd, km, qm, kId);
#pragma unroll
              for (int kk = 1; kk < D / 32; ++kk) mma_e4m3<true>(sd, km + kk * 2, qm + kk * 2, kId);
              tc_commit(done);
            }
            __syncwarp();
            if (++s == C::kKSt) {
              s = 0;
              ++lap;
            }
          }
        }
        if (ok && el) tc_commit(bar_at(B->q_empty, m & 1));
        __syncwarp();
      }
    } else {
      constexpr uint32_t kId = idesc_e4m3(kPos, 2 * NP, true, true);
      // MN-major operands: strides between atoms along M / N and between groups of 8 positions
      const uint64_t vd = sdesc(sb + C::kVOff, kTileBytes, 1024, 2);
      const uint64_t pd = sdesc(sb + C::kPOff, C::kPTile, 8 * C::kPRow, C::kPSwz);
#pragma unroll 1
      for (int m = 0; ok; ++m) {
        Span x;
        if (!ring_span(m, x)) break;
        const int tb = uni(x.t0), te = uni(x.t1);
#pragma unroll 1
        for (int t0 = tb; t0 < te && ok; t0 += C::kMT, ++n) {
          if (n >= 2 && !waitb(&B->o_empty[n & 1], (n - 2) >> 1)) {
            ok = false;
            break;
          }
          const uint32_t od = tmem + (n & 1) * 2 * NP;
          const int t1 = min(t0 + C::kMT, te);
#pragma unroll 1
          for (int t = t0; t < t1; ++t, ++g) {
            const int s = g % C::kVSt;   // V stage and P^T slot
            if (!waitb(&B->vfull[s], g / C::kVSt) || !waitb(&B->pfull[s], g / C::kPT)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t vm = vd + s * (kTileBytes >> 4), pm = pd + s * (C::kPTile >> 4);
            const uint32_t done = bar_at(B->pvd, s);
            if (t == t0) {
              if (el) mma_e4m3<false>(od, vm, pm, kId);
            } else {
              if (el) mma_e4m3<true>(od, vm, pm, kId);
            }
            if (el) {
#pragma unroll
              for (int kk = 1; kk < kPos / 32; ++kk)
                mma_e4m3<true>(od, vm + kk * (32 * 128 >> 4), pm + kk * (32 * C::kPRow >> 4), kId);
              tc_commit(done);
            }
            __syncwarp();
          }
          if (ok && el) tc_commit(bar_at(B->o_full, n & 1));
          __syncwarp();
        }
      }
    }
    if (el) tc_commit(smem_u32(&B->fin[warp & 1]));
    __syncwarp();
    mbar_wait(smem_u32(&B->fin[warp & 1]), 0);   // not cut short by an abort: the work is in flight
  } else if (warp < kPWarp0) {
    // =================================================================== first pass ====
    const int q4 = warp & 3;                        // tensor-memory lane quarter
    const int lrow = q4 * 32 + lane;                // tile position of this thread
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
    uint32_t wg_phase = 0;
    // lane j keeps the running reference of row j (half j / NR); the four warps hold the same values
    float mrun = 0.f;
    const int jl = lane < 2 * NR ? lane : 2 * NR - 1, jc = jl / NR * NH + jl % NR;   // row, its column
    bool ok = true;
    int n = 0, g = 0, s = 0, lap = 0;   // chunks, tiles; position in the K ring
#pragma unroll 1
    for (int m = 0; ok && !aborted(abort_flag); ++m) {
      Span x;
      if (!ring_span(m, x)) break;
      const int L = x.L, Lc = x.L + T;
      const int rows = min(p.Rg, R - x.g0);
      float* scores = CAP && p.scores ? p.scores + (((size_t)x.r * Hkv + x.kvh) * R + x.g0) * (size_t)p.cap : nullptr;
      const float* rsm = rs + (m & 7) * NP;
#pragma unroll 1
      for (int t0 = x.t0; t0 < x.t1; t0 += C::kMT, ++n) {
        const int nt = min(C::kMT, x.t1 - t0);
        // the chunk's page scales; its logits' buffer (with the first tile: the span's row factors)
        if (!waitb(&B->sc_full[n & (kScaleBufs - 1)], n / kScaleBufs) ||
            (n >= 2 && !waitb(&B->x_empty[n & 1], (n - 2) >> 1))) {
          ok = false;
          break;
        }
        const float* ksc = scs + (n & (kScaleBufs - 1)) * kScaleFloats + (lrow >> 4);   // + 8 per tile
        const float* lvc = ksc + 128;
        float2 mrow[2 * RP];
#pragma unroll
        for (int j = 0; j < 2 * RP; ++j) mrow[j] = make_float2(-INFINITY, -INFINITY);
#pragma unroll 1
        for (int u = 0; u < nt; ++u, ++g) {
          const int d = g % C::kNS;
          if (!waitb(&B->qkd[s], lap)) {
            ok = false;
            break;
          }
          if (++s == C::kKSt) {
            s = 0;
            ++lap;
          }
          tc_fence_after();
          float v[2][NP];   // per half of the rows: NH of qh, NH of ql
          tmem_ld<NP>(tl + C::kSCol0 + d * 2 * NP, v[0]);
          tmem_ld<NP>(tl + C::kSCol0 + d * 2 * NP + NP, v[1]);
          tmem_wait_ld();
          tmem_tie(v[0]);
          tmem_tie(v[1]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&B->sempty[d]));
          const int p0 = (t0 + u) * kPos, pos = p0 + lrow;
          const float ks = ksc[u * 8], lv = lvc[u * 8];
          const float2 ks2 = make_float2(ks, ks), lv2 = make_float2(lv, lv);
          // masked: the tile holds positions that some row does not see (compiled apart without capture,
          // so that the other tiles' code is straight; with capture one copy is faster)
          auto take = [&](auto m_) {
            const bool masked = m_;
            // the first row that sees the position: pos - L <= its block row
            const int r0 = pos < L ? 0 : (pos < Lc ? (pos - L) * G - x.g0 : kPos);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float2 y[RP];
#pragma unroll
              for (int j = 0; j < RP; ++j)
                y[j] = mul2(mul2(add2(make_float2(v[h][2 * j], v[h][2 * j + 1]),
                                      make_float2(v[h][NH + 2 * j], v[h][NH + 2 * j + 1])), ks2),
                            *reinterpret_cast<const float2*>(rsm + h * NH + 2 * j));
              if (scores && pos < L) {
                // a warp's 32 lanes write 32 consecutive positions of a row, one whole 128-byte line
                float* srow = scores + (size_t)(h * NR) * p.cap + pos;
#pragma unroll
                for (int j = 0; j < RP; ++j) {
                  if (h * NR + 2 * j < rows) *srow = y[j].x * kLn2;
                  srow += p.cap;
                  if (h * NR + 2 * j + 1 < rows) *srow = y[j].y * kLn2;
                  srow += p.cap;
                }
              }
              if (masked) {
#pragma unroll
                for (int j = 0; j < RP; ++j) {
                  if (h * NR + 2 * j < r0) y[j].x = -INFINITY;
                  if (h * NR + 2 * j + 1 < r0) y[j].y = -INFINITY;
                }
              }
              float xo[NH];
#pragma unroll
              for (int j = 0; j < NH; ++j) xo[j] = j < NR ? ((j & 1) ? y[j / 2].y : y[j / 2].x) : 0.f;
              tmem_st(tl + C::kXCol0 + ((n & 1) * C::kMT + u) * NP + h * NH, xo);
#pragma unroll
              for (int j = 0; j < RP; ++j) {
                const float2 z = add2(y[j], lv2);
                mrow[h * RP + j].x = fmaxf(mrow[h * RP + j].x, z.x);
                mrow[h * RP + j].y = fmaxf(mrow[h * RP + j].y, z.y);
              }
            }
          };
          if constexpr (CAP) take(p0 + kPos > L);
          else if (__builtin_expect(p0 + kPos > L, 0)) take(std::true_type{});
          else take(std::false_type{});
        }
        tmem_wait_st();
        tc_fence_before();
        if (!ok) break;
        {
          float mx[2 * NR];
#pragma unroll
          for (int j = 0; j < 2 * NR; ++j) mx[j] = (j & 1) ? mrow[j / 2].y : mrow[j / 2].x;
          const float r = ColReduce<2 * NR>::run(mx, lane, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
          const int c = ColReduce<2 * NR>::col_of(lane);
          if (c < 2 * NR) redM[((n & 1) * 4 + q4) * NP + c] = r;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&B->wg[2]));
        if (!waitb(&B->wg[2], wg_phase)) {
          ok = false;
          break;
        }
        wg_phase ^= 1u;
        const float* m4 = redM + (n & 1) * 4 * NP + jl;
        const float mc = fmaxf(fmaxf(m4[0], m4[NP]), fmaxf(m4[2 * NP], m4[3 * NP])) - 8.f;
        const bool first = t0 == x.t0;
        const float mn = first ? mc : fmaxf(mrun, mc);
        if (q4 == 0 && lane < 2 * NR) {
          float* rf = refs + (n & 3) * 3 * NP + jc;
          rf[0] = mn == -INFINITY ? 0.f : -mn;   // nothing seen yet: 2^-inf = 0
          rf[NP] = first || mrun == -INFINITY ? 0.f : exp2f(0.5f * (mrun - mn));
          rf[2 * NP] = mn;
        }
        mrun = mn;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&B->x_full[n & 1]));
      }
    }
  } else {
    // ================================================================== second pass ====
    const int sg = (warp - kPWarp0) >> 2;           // warpgroup: rows [sg NR, sg NR + NR)
    const int q4 = warp & 3;
    const int lrow = q4 * 32 + lane;                // tile position (x) or d (O) of this thread
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
    // 16-byte chunk XOR of this position's P^T row (32-, 64-byte swizzle)
    const int swz_row = NP == 16 ? ((lrow >> 2) & 1) : ((lrow >> 1) & 3);
    // The first span's q rows, by all eight warps: the K producer, which splits the later spans' while
    // their predecessors stream, is 4 us about 28 rows (4 requests of 40 tokens: 19.2 us by it, 14.8
    // so, 15.7 by the first pass's four warps; 32 requests of 8K to 24K 371, 360 and 370).
    {
      Span x;
      if (ring_span(0, x)) {
        const int rows = min(p.Rg, R - x.g0), j = (warp - kPWarp0) * RI + lane / LR;
        constexpr int kTimes = (2 * NR + kPWarps * RI - 1) / (kPWarps * RI);
        uint4 raw[kTimes];
#pragma unroll
        for (int i = 0; i < kTimes; ++i) raw[i] = load_q(x, j + i * kPWarps * RI, rows);
#pragma unroll
        for (int i = 0; i < kTimes; ++i) split_row(raw[i], j + i * kPWarps * RI, rows, 0);
        if (warp == kPWarp0) zero_factors(rows, 0);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&B->q0));
      }
    }
    uint32_t wg_phase = 0;
    float orun[NR], lsum[NR];   // O of the span (this thread's d) and row sums, relative to the reference
    // Chunk n's O joins the span; with its last chunk the span's record (or, when the span is the
    // whole context, the output) is written.
    auto epilogue = [&](int n, int m, bool first, bool last, float ov) -> bool {
      if (last) {   // the sums of the group's warps are there
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&B->wg[sg]));
        if (!waitb(&B->wg[sg], wg_phase)) return false;
        wg_phase ^= 1u;
      }
      if (!waitb(&B->o_full[n & 1], n >> 1)) return false;
      tc_fence_after();
      float o[NP];
      tmem_ld<NP>(tl + (n & 1) * 2 * NP + sg * NP, o);
      tmem_ready(o);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&B->o_empty[n & 1]));
      const float* rf = refs + (n & 3) * 3 * NP + sg * NH;
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const float v = fmaf(o[NH + j], 0.03125f, o[j]) * ov;
        orun[j] = first ? v : fmaf(orun[j], rf[NP + j] * rf[NP + j], v);
      }
      if (!last) return true;
      Span x;
      read_span(m, x);
      const int rows = min(NR, min(p.Rg, R - x.g0) - sg * NR), row0 = x.g0 + sg * NR;
      const float* rl4 = redL + (m & 1) * 8 * NH + sg * 4 * NH;   // sums of the group's warps
      if (x.nsp == 1) {
#pragma unroll 1
        for (int j = 0; j < rows; ++j) {   // (a loop: its code would otherwise be a quarter of the kernel)
          float o = 0.f;
#pragma unroll
          for (int i = 0; i < NR; ++i)
            if (i == j) o = orun[i];
          const float l = (rl4[j] + rl4[NH + j]) + (rl4[2 * NH + j] + rl4[3 * NH + j]);
          const int t = (row0 + j) / G, gq = row0 + j - t * G;
          const size_t orow = ((size_t)x.r * T + t) * p.Hq + x.kvh * G + gq;
          if (lrow < D) p.out[orow * D + lrow] = __float2bfloat16_rn(o / l);
          if (lrow == 0) p.lse[orow] = (rf[2 * NP + j] + log2f(l)) * kLn2;
        }
        return true;
      }
      float* rec = p.part + (size_t)x.id * p.Rp * (D + 2);
      if (lrow < D) {
#pragma unroll
        for (int j = 0; j < NR; ++j)
          if (j < rows) rec[2 * p.Rp + (size_t)(sg * NR + j) * D + lrow] = orun[j];
      }
      if (q4 == 0 && lane < rows) {
        rec[sg * NR + lane] = rf[2 * NP + lane];
        rec[p.Rp + sg * NR + lane] = (rl4[lane] + rl4[NH + lane]) + (rl4[2 * NH + lane] + rl4[3 * NH + lane]);
      }
      return true;
    };

    bool ok = true;
    int n = 0, gs = 0;          // chunks, tiles
    float ovp = 0.f;            // of the chunk before: unit of V scales, span, place in it
    int mp = 0;
    bool pfirst = false, plast = false;
#pragma unroll 1
    for (int m = 0; ok && !aborted(abort_flag); ++m) {
      Span x;
      if (!ring_span(m, x)) break;
#pragma unroll 1
      for (int t0 = x.t0; t0 < x.t1; t0 += C::kMT, ++n) {
        const int nt = min(C::kMT, x.t1 - t0);
        const bool first = t0 == x.t0, last = t0 + nt == x.t1;
        if (!waitb(&B->x_full[n & 1], n >> 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float* vsc = scs + (n & (kScaleBufs - 1)) * kScaleFloats + 64 + (lrow >> 4);   // + 8 per tile
        const float* rf = refs + (n & 3) * 3 * NP + sg * NH;
        const uint32_t xb = tl + C::kXCol0 + (n & 1) * C::kMT * NP + sg * NH;
        float v[NH];
        tmem_ld<NH>(xb, v);
        float2 nm[RP];
#pragma unroll
        for (int j = 0; j < RP; ++j) {
          nm[j] = *reinterpret_cast<const float2*>(rf + 2 * j);
          const float2 f = *reinterpret_cast<const float2*>(rf + NP + 2 * j);
          const float2 ls = mul2(mul2(make_float2(lsum[2 * j], lsum[2 * j + 1]), f), f);
          lsum[2 * j] = first ? 0.f : ls.x;
          lsum[2 * j + 1] = first ? 0.f : ls.y;
        }
        // 2^(x - m), its sum in fp32, times vs / vref in two e4m3 parts to P^T. The next tile's logits
        // are on their way while this one is worked on, and a tile's P^T is handed over once the
        // next one is ready to be stored (its stores have drained by then).
        auto publish = [&](int slot) {
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&B->pfull[slot]));
        };
#pragma unroll 1
        for (int u = 0; u < nt; ++u, ++gs) {
          tmem_ready(v);
          float2 e[RP];
#pragma unroll
          for (int j = 0; j < RP; ++j) e[j] = add2(make_float2(v[2 * j], v[2 * j + 1]), nm[j]);
          if (u + 1 < nt) tmem_ld<NH>(xb + (u + 1) * NP, v);
          const float vw = vsc[u * 8];
          const float2 vw2 = make_float2(vw, vw);
          uint32_t all[NP / 4];
#pragma unroll
          for (int j = 0; j < NP / 4; ++j) all[j] = 0;
#pragma unroll
          for (int j = 0; j < RP; ++j) {
            e[j] = make_float2(ex2(e[j].x), ex2(e[j].y));
            const float2 ls = add2(make_float2(lsum[2 * j], lsum[2 * j + 1]), e[j]);
            lsum[2 * j] = ls.x;
            lsum[2 * j + 1] = ls.y;
            uint32_t h, l;
            split_e4m3x2(mul2(e[j], vw2), h, l);
            // this warpgroup's NP bytes of the position's row: NH bytes of ph, then NH of pl
            uint32_t &hw = all[j / 2], &lw = all[NH / 4 + j / 2];
            hw = (j & 1) ? __byte_perm(hw, h, 0x5410) : h;
            lw = (j & 1) ? __byte_perm(lw, l, 0x5410) : l;
          }
          const int slot = gs % C::kPT;
          if (u > 0) publish((gs - 1) % C::kPT);
          if (gs >= C::kPT && !waitb(&B->pvd[slot], gs / C::kPT - 1)) {
            ok = false;
            break;
          }
          uint8_t* ptile = smem + C::kPOff + slot * C::kPTile + lrow * C::kPRow;
#pragma unroll
          for (int i = 0; i < NP / 16; ++i)
            *reinterpret_cast<uint4*>(ptile + (((sg * (NP / 16) + i) ^ swz_row) << 4)) =
                make_uint4(all[4 * i], all[4 * i + 1], all[4 * i + 2], all[4 * i + 3]);
        }
        if (!ok) {
          tmem_wait_ld();   // nothing in flight when the tensor memory goes away
          break;
        }
        const float vref = scs[(n & (kScaleBufs - 1)) * kScaleFloats + 192];
        tc_fence_before();
        publish((gs - 1) % C::kPT);
        if (lane == 0) {
          mbar_arrive(smem_u32(&B->x_empty[n & 1]));
          mbar_arrive(smem_u32(&B->sm_done[n & (kScaleBufs - 1)]));
        }
        // the previous chunk's O (its PV has had this chunk's pass to finish)
        if (n > 0 && !epilogue(n - 1, mp, pfirst, plast, ovp)) {
          ok = false;
          break;
        }
        if (last) {
          const float r = ColReduce<NR>::run(lsum, lane, 0.f, [](float a, float b) { return a + b; });
          const int c = ColReduce<NR>::col_of(lane);
          if (c < NR) redL[((m & 1) * 8 + sg * 4 + q4) * NH + c] = r;   // read behind the epilogue's barrier
        }
        mp = m;
        pfirst = first;
        plast = last;
        ovp = vref;
      }
    }
    if (ok && n > 0 && !aborted(abort_flag)) epilogue(n - 1, mp, pfirst, plast, ovp);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // the last CTA out returns the counters to zero for the next launch
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(p.sched + 1, 1) == (int)gridDim.x - 1) {
      p.sched[0] = 0;
      p.sched[1] = 0;
    }
  }
}

// Joins the span records of every (request, KV head) that has more than one: a warp per row,
// out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, spans in order (nothing depends on which
// CTA finished first). The records were just written, so they come from L2.
constexpr int kMergeWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kv8_kernel(const VerifyKv8Params p, int batch) {
  pdl_wait();
  constexpr int V = D / 32;   // consecutive d of a lane
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kMergeWarps + (threadIdx.x >> 5), kvh = blockIdx.y, bl = blockIdx.z;
  if (row >= p.R) return;
  const int r = p.req_ids ? p.req_ids[p.req_off + bl] : p.req_off + bl;
  if (r < 0 || r >= p.num_requests) return;      // reported by the attention kernel
  const int b0 = p.plan[1 + bl], b1 = p.plan[2 + bl];
  const int nsp = (b1 - b0) / (p.Hkv * p.ngroups);
  if (nsp <= 1) return;                          // no work, or written by the attention kernel
  const int grp = row / p.Rg, jr = row - grp * p.Rg;   // the records are those of the row's group
  const size_t one = (size_t)p.Rp * (D + 2), pitch = one * p.ngroups;
  const float* rec = p.part + ((size_t)b0 + (size_t)kvh * nsp * p.ngroups + grp) * one;
  float M = -INFINITY;
  for (int s = lane; s < nsp; s += 32) M = fmaxf(M, __ldcg(rec + s * pitch + jr));
  M = warp_max(M);
  float lsum = 0.f;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (int s0 = 0; s0 < nsp; s0 += 32) {
    float h = 0.f, l = 0.f;   // root of the weight: see kMaxRatio
    if (s0 + lane < nsp) {
      const float ms = __ldcg(rec + (s0 + lane) * pitch + jr);
      l = __ldcg(rec + (s0 + lane) * pitch + p.Rp + jr);
      h = ms == -INFINITY ? 0.f : exp2f(0.5f * (ms - M));
    }
    lsum = fmaf(h, h * l, lsum);
    const float w = h * h;
    const int cnt = min(32, nsp - s0);
    const float* o = rec + s0 * pitch + 2 * p.Rp + (size_t)jr * D + lane * V;
    int u = 0;
    for (; u + 4 <= cnt; u += 4) {
      float x[4][V];
#pragma unroll
      for (int q = 0; q < 4; ++q) ld_vec<V>(o + (u + q) * pitch, x[q]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float wq = __shfl_sync(kFull, w, u + q);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(wq, x[q][i], acc[i]);
      }
    }
    for (; u < cnt; ++u) {
      float x[V];
      ld_vec<V>(o + u * pitch, x);
      const float wq = __shfl_sync(kFull, w, u);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(wq, x[i], acc[i]);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) lsum += __shfl_xor_sync(kFull, lsum, o);
  const int t = row / p.G, gq = row - t * p.G;
  const size_t orow = ((size_t)r * p.T + t) * p.Hq + kvh * p.G + gq;
  __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(p.out + orow * D + lane * V);
#pragma unroll
  for (int i = 0; i < V; i += 2) dst[i / 2] = __floats2bfloat162_rn(acc[i] / lsum, acc[i + 1] / lsum);
  if (lane == 0) p.lse[orow] = (M + log2f(lsum)) * kLn2;
}

}  // namespace kv8

template <int RP, int D, bool CAP>
static int launch_kv8_c(const CUtensorMap& k1, const CUtensorMap& v1, const CUtensorMap& k8,
                        const CUtensorMap& v8, const VerifyKv8Params& p, int batch, int num_sms,
                        cudaStream_t stream) {
  using C = kv8::Cfg<RP>;
  static std::atomic<uint64_t> attr_done{0};
  if (cuda_status(ensure_smem_attr(kv8::verify_kv8_kernel<RP, D, CAP>, C::kSmem, attr_done), "cudaFuncSetAttribute") != S3R_OK)
    return S3R_ERR_CUDA;
  launch_pdl(kv8::verify_kv8_kernel<RP, D, CAP>, num_sms, kv8::kThreads, C::kSmem, stream, k1, v1, k8, v8, p, batch);
  return cuda_status(cudaGetLastError(), "s3r_verify_attn_kv8");
}

template <int RP, int D>
static int launch_kv8_t(const CUtensorMap& k1, const CUtensorMap& v1, const CUtensorMap& k8,
                        const CUtensorMap& v8, const VerifyKv8Params& p, int batch, int num_sms,
                        cudaStream_t stream) {
  return p.scores ? launch_kv8_c<RP, D, true>(k1, v1, k8, v8, p, batch, num_sms, stream)
                  : launch_kv8_c<RP, D, false>(k1, v1, k8, v8, p, batch, num_sms, stream);
}

template <int D>
static int launch_kv8_d(const CUtensorMap& k1, const CUtensorMap& v1, const CUtensorMap& k8,
                        const CUtensorMap& v8, const VerifyKv8Params& p, int batch, int num_sms,
                        cudaStream_t stream) {
  int st;
  // Pairs of rows per warpgroup, up to the next instance. Up to 4 pairs (16 rows) an instance is worth
  // little without capture and up to 3 % with it: 4 rows take 181 us (196 with capture) in instance 1 and
  // 183 (200) in 4, 8 rows 183 (206) in 2 and 186 (212) in 4, 12 rows 189 (222) in 4 and 187 (220) in one of
  // their own, which is not built. Above, each is: 16 rows 191 (234) in 4 and 239 (278) in 5, 20 rows
  // 254 (296) in 5 and 280 (333) in 7, 28 rows 298 (362) in 7 and 302 (460) in 8. An instance for 24 rows
  // would take 280 (318) where 7 takes 290 (348); it is not built either.
  // (32 requests of 8K to 24K tokens, 8 heads of 128, one B200.)
  const int rp = (p.Rg + 3) / 4;
  if (rp <= 1) st = launch_kv8_t<1, D>(k1, v1, k8, v8, p, batch, num_sms, stream);
  else if (rp <= 2) st = launch_kv8_t<2, D>(k1, v1, k8, v8, p, batch, num_sms, stream);
  else if (rp <= 4) st = launch_kv8_t<4, D>(k1, v1, k8, v8, p, batch, num_sms, stream);
  else if (rp <= 5) st = launch_kv8_t<5, D>(k1, v1, k8, v8, p, batch, num_sms, stream);
  else if (rp <= 7) st = launch_kv8_t<7, D>(k1, v1, k8, v8, p, batch, num_sms, stream);
  else st = launch_kv8_t<8, D>(k1, v1, k8, v8, p, batch, num_sms, stream);
  if (st != S3R_OK) return st;
  dim3 grid((p.R + kv8::kMergeWarps - 1) / kv8::kMergeWarps, p.Hkv, batch);
  launch_pdl(kv8::merge_kv8_kernel<D>, grid, 32 * kv8::kMergeWarps, 0, stream, p, batch);
  return cuda_status(cudaGetLastError(), "s3r_verify_attn_kv8 merge");
}

int verify_kv8_groups(int R) { return R > 32 ? 2 : 1; }

int launch_verify_kv8(const CUtensorMap& k1, const CUtensorMap& v1, const CUtensorMap& k8,
                      const CUtensorMap& v8, const VerifyKv8Params& p, int D, int batch, int num_sms,
                      cudaStream_t stream, int* launches) {
  *launches = 0;
  for (int b0 = 0; b0 < batch; b0 += kv8::kMaxBatch) {
    VerifyKv8Params q = p;
    q.req_off = b0;
    const int nb = batch - b0 < kv8::kMaxBatch ? batch - b0 : kv8::kMaxBatch;
    const int st = D == 128 ? launch_kv8_d<128>(k1, v1, k8, v8, q, nb, num_sms, stream)
                            : launch_kv8_d<64>(k1, v1, k8, v8, q, nb, num_sms, stream);
    if (st != S3R_OK) return st;
    *launches += 2;
  }
  return S3R_OK;
}

// Plan area and span records of one launch (at most kMaxBatch requests): the span length is
// at least total tiles / (6 spans per SM) (or covers a chunk), so there are at most 6 spans per
// SM and one more for each (request, KV head, row group).
size_t verify_kv8_bytes(int num_requests, int Hkv, int R, int D, int num_sms) {
  const int nb = num_requests < kv8::kMaxBatch ? num_requests : kv8::kMaxBatch;
  const int ng = verify_kv8_groups(R);
  const size_t spans = (size_t)nb * Hkv * ng + (size_t)kSpansPerCta * num_sms;
  return kv8::kPlanInts * 4 + align_up(spans * (size_t)verify_kv8_rec_rows((R + ng - 1) / ng) * (D + 2) * 4, 256);
}

int verify_kv8_rec_rows(int Rg) { return (Rg + 3) / 4 * 4; }
int verify_kv8_plan_bytes() { return kv8::kPlanInts * 4; }

}  // namespace s3r
