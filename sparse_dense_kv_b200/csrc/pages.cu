// Page tables and slot maps on the GPU: pages from a free stack for the requests' next tokens,
// and back to it.
//
// What they compute, requests in batch order b: with need_b the pages the request shall hold,
//   allocation: add_b = max(0, need_b - held_b), before_b = sum_{b' < b} add_b'; the request is
//     served iff before_b + add_b <= free_count (or add_b = 0), and its i-th new page is
//     free_pages[free_count - 1 - before_b - i];
//   release: gone_b = max(0, held_b - need_b), and its i-th page goes to
//     free_pages[free_count + before_b + i].
// So the result depends on nothing but the inputs.
//
// Bound: latency for a round's few pages (one launch, two dependent loads deep), HBM writes
// (8 bytes per slot) when prompts are admitted. A CTA takes `rp` requests and a segment of their
// slots (pages, when releasing); it sums the demand of all earlier requests itself, which the
// L2 serves (a few hundred CTAs x a few bytes per request), instead of a scan launch before it.
// Measured: a round of 32 requests 7.4 us, 256 prompts of up to 16k tokens with their slot map 14 to
// 17 us (33 MB of slots; 22.5 us with one slot per store), release of a ragged batch of 256 8.2 us.
// held_out and free_count_out may be held and free_count themselves: only the last CTA to finish
// writes them.
#include "kernels.h"
#include "kv8.cuh"

namespace s3r {

constexpr int kPagesThreads = 256;
constexpr int kAllocSeg = 4096;      // slots of a CTA's segment
constexpr int kReleaseSeg = 1024;    // pages of a CTA's segment

constexpr int kEmpty = -2;
struct PageDemand {
  int r;         // request; kEmpty, or -1 if its id is out of range
  int L, n;      // committed length, tokens (release: 0)
  int held, need, delta;   // pages held and wanted, demand
  bool bad;      // an input out of range: nothing changes hands
};

template <bool RELEASE>
__device__ __forceinline__ PageDemand demand_of(const PagesParams& p, int b) {
  PageDemand d{};
  d.r = p.req_ids ? p.req_ids[b] : b;
  if (d.r < 0 || d.r >= p.num_requests) {
    d.r = d.r == S3R_NO_REQUEST ? kEmpty : -1;
    d.bad = true;
    return d;
  }
  d.held = p.held[d.r];
  int64_t upto;
  if (RELEASE) {
    upto = p.keep_len ? p.keep_len[d.r] : 0;
    d.bad = upto < 0;
  } else {
    d.L = p.seq_lens[d.r];
    d.n = p.n_new ? p.n_new[d.r] : p.T;
    d.bad = d.L < 0 || d.n < 0 || d.n > p.T;
    upto = (int64_t)d.L + d.n;
  }
  const int64_t pages = (upto + kPage - 1) / kPage;
  d.bad = d.bad || d.held < 0 || d.held > p.max_pages || (!RELEASE && pages > p.max_pages);
  if (!d.bad) {
    d.need = (int)(pages < p.max_pages ? pages : p.max_pages);
    d.delta = RELEASE ? max(0, d.held - d.need) : max(0, d.need - d.held);
  }
  return d;
}

// Exclusive sum over the CTA's threads; `total` receives the whole sum.
__device__ __forceinline__ long long block_exclusive(long long v, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();   // warp_sums is free again
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPagesThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  return before + incl - v;
}

template <bool RELEASE>
__global__ void __launch_bounds__(kPagesThreads) pages_kernel(const PagesParams p) {
  pdl_wait();
  __shared__ long long warp_sums[kPagesThreads / 32];
  __shared__ PageDemand dem[kPagesThreads];
  __shared__ long long before_s[kPagesThreads];
  __shared__ int s_flag;
  const int tid = threadIdx.x;
  const int b0 = blockIdx.y * p.rp, nb = min(p.rp, p.batch - b0);
  const long long have = p.free_count[0];
  // what may change hands in all: the stack's pages, or the room above them
  const long long limit = RELEASE ? (have < 0 || have > p.free_capacity ? -1 : p.free_capacity - have)
                                  : (have < 0 || have > p.free_capacity ? -1 : have);
  // demand of the requests before this CTA's
  long long mine = 0;
  for (int b = tid; b < b0; b += kPagesThreads) mine += demand_of<RELEASE>(p, b).delta;
  long long base;
  block_exclusive(mine, warp_sums, base);
  PageDemand d{};
  if (tid < nb) d = demand_of<RELEASE>(p, b0 + tid);
  long long total;
  const long long before = base + block_exclusive(tid < nb ? d.delta : 0, warp_sums, total);
  if (tid < nb) {
    // not served: keeps what it has
    if (d.bad || (d.delta > 0 && before + d.delta > limit)) {
      if (blockIdx.x == 0 && d.r != kEmpty && (d.bad || RELEASE)) set_error(p.err, S3R_ERR_DEVICE_BOUNDS);
      d.bad = true;
      d.delta = 0;
    }
    dem[tid] = d;
    before_s[tid] = before;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0 && limit < 0) set_error(p.err, S3R_ERR_DEVICE_BOUNDS);
  __syncthreads();

  // pages change hands: with many requests in the CTA each has few pages (rp is chosen so) and a
  // thread takes a request; with few, all threads take one request after the other
  const bool many = p.rp >= 16;
  const int j0 = many ? (int)blockIdx.x : (int)blockIdx.x * kPagesThreads + tid;
  const int dj = many ? (int)gridDim.x : (int)gridDim.x * kPagesThreads;
  for (int i = many ? tid : 0; i < nb; i += many ? kPagesThreads : 1) {
    const PageDemand x = dem[i];
    if (x.r < 0) continue;
    int32_t* row = p.page_table + (size_t)x.r * p.max_pages;
    for (int j = j0; j < x.delta; j += dj) {
      if (RELEASE) p.free_pages[have + before_s[i] + j] = row[x.need + j];
      else row[x.held + j] = p.free_pages[have - 1 - before_s[i] - j];
    }
  }
  if (!RELEASE && p.slot_map) {
    const int t0 = blockIdx.x * kAllocSeg, seg = min(kAllocSeg, p.T - t0);
    // the slot of a request's token t; -1 where it has none
    auto slot_of = [&](const PageDemand& x, long long top, int t) -> int64_t {
      if (x.bad || t >= x.n) return -1;
      const uint32_t pos = (uint32_t)(x.L + t);
      const int pg = (int)(pos / kPage);
      const int page = pg < x.held ? p.page_table[(size_t)x.r * p.max_pages + pg] : p.free_pages[top - pg];
      return (int64_t)page * kPage + pos % kPage;
    };
    if (p.T >= 2 * kPagesThreads) {
      // long rows: two slots per store where the row's address allows it, four stores in flight
      for (int i = 0; i < nb; ++i) {
        const PageDemand x = dem[i];
        if (x.r < 0) continue;
        const long long top = have - 1 - before_s[i] + x.held;
        int64_t* row = p.slot_map + (size_t)x.r * p.T + t0;
        const int odd = (int)(((uintptr_t)row >> 3) & 1);
        const int pairs = (seg - odd) / 2;
        if (tid == 0 && odd) row[0] = slot_of(x, top, t0);
        if (tid == 0 && odd + 2 * pairs < seg) row[seg - 1] = slot_of(x, top, t0 + seg - 1);
        longlong2* out = reinterpret_cast<longlong2*>(row + odd);
#pragma unroll 4
        for (int k = tid; k < pairs; k += kPagesThreads) {
          const int t = t0 + odd + 2 * k;
          out[k] = make_longlong2(slot_of(x, top, t), slot_of(x, top, t + 1));
        }
      }
    } else {
      // short rows, flattened over the CTA's requests
      for (int k = tid; k < nb * seg; k += kPagesThreads) {
        const int i = k / seg, t = t0 + k - i * seg;
        const PageDemand& x = dem[i];
        if (x.r < 0) continue;
        p.slot_map[(size_t)x.r * p.T + t] = slot_of(x, have - 1 - before_s[i] + x.held, t);
      }
    }
  }

  if (!last_of(p.ticket, gridDim.x * gridDim.y, &s_flag)) return;
  // the last CTA: every input has been read
  long long run = 0, taken = 0;
  for (int c0 = 0; c0 < p.batch; c0 += kPagesThreads) {
    const int b = c0 + tid;
    PageDemand y{};
    if (b < p.batch) y = demand_of<RELEASE>(p, b);
    long long sum, moved;
    const long long bef = run + block_exclusive(b < p.batch ? y.delta : 0, warp_sums, sum);
    const bool served = b < p.batch && !y.bad && (y.delta == 0 || bef + y.delta <= limit);
    block_exclusive(served ? y.delta : 0, warp_sums, moved);   // (a barrier: `held` of this batch of requests has been read)
    if (b < p.batch && y.r >= 0) {
      p.held_out[y.r] = served ? y.held + (RELEASE ? -y.delta : y.delta) : y.held;
      if (!RELEASE) p.granted[y.r] = served ? 1 : 0;
    }
    run += sum;
    taken += moved;
  }
  if (tid == 0) p.free_count_out[0] = (int)(RELEASE ? have + taken : have - taken);
}

// Requests per CTA: up to 4096 slots (1024 pages, when releasing) of work each.
int launch_alloc_pages(const PagesParams& p0, cudaStream_t stream) {
  PagesParams p = p0;
  p.rp = p.T > 0 ? kAllocSeg / p.T : kPagesThreads;
  p.rp = p.rp < 1 ? 1 : (p.rp > kPagesThreads ? kPagesThreads : p.rp);
  const int most = 65535;   // grid.y
  if ((p.batch + p.rp - 1) / p.rp > most) return S3R_ERR_UNSUPPORTED;
  dim3 grid(p.T > kAllocSeg ? (p.T + kAllocSeg - 1) / kAllocSeg : 1, (p.batch + p.rp - 1) / p.rp);
  launch_pdl(pages_kernel<false>, grid, kPagesThreads, 0, stream, p);
  return cuda_status(cudaGetLastError(), "s3r_alloc_pages");
}

int launch_release_pages(const PagesParams& p0, cudaStream_t stream) {
  PagesParams p = p0;
  p.rp = kReleaseSeg / p.max_pages;
  p.rp = p.rp < 1 ? 1 : (p.rp > kPagesThreads ? kPagesThreads : p.rp);
  dim3 grid((p.max_pages + kReleaseSeg - 1) / kReleaseSeg, (p.batch + p.rp - 1) / p.rp);
  launch_pdl(pages_kernel<true>, grid, kPagesThreads, 0, stream, p);
  return cuda_status(cudaGetLastError(), "s3r_release_pages");
}

}  // namespace s3r
