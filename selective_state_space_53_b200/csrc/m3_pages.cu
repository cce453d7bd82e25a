// m3_pages.cu -- pages of a pool of recurrent states: copy, fork, free, compact.
//
// A page is row i of every buffer of the pool (each layer's h, carry_B and carry_x, say).  The copy
// kernel gives every thread one 16-byte lane of the page, fixed for the whole list of moves, and
// takes the list in order: no two threads touch the same bytes, so the list acts as one move after
// the other whatever pages it names twice.  Four moves are in flight per thread: their loads are
// issued together, and a load whose page an earlier move of the four writes takes that move's value
// from its register instead.  Bound by HBM (a page is read and written once per move): moving 72 pages of
// 8.7 MB takes 189 us (6.4 TB/s), forking 24 of them 63 us (6.7 TB/s).
#include "m3_linattn.cuh"

namespace m3 {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kMoves = 4;  // moves in flight per thread

struct CopyPlan {
  int nbuf;
  int npages;
  uint32_t first[M3_PAGES_MAX_BUF + 1];  // first block of each buffer
  uint4* base[M3_PAGES_MAX_BUF];
  int64_t lanes[M3_PAGES_MAX_BUF];       // 16-byte lanes of a page
};

// moves [0, n) of (src, dst); null dst: the destination is the move's own index.  range (may be
// null): moves [range[1], range[0]).  zero_neg: a negative source writes zeros (otherwise the move
// is skipped).  The moves are split over gridDim.y only when the caller knows them independent.
__global__ void __launch_bounds__(kCopyThreads)
    pages_copy_kernel(const __grid_constant__ CopyPlan pl, int64_t n, const int32_t* src, const int32_t* dst,
                      const int32_t* range, int zero_neg, int* status) {
  int lo = 0, hi = pl.nbuf - 1;
  while (lo < hi) {  // the last buffer that starts at or before this block
    const int mid = (lo + hi + 1) >> 1;
    if (pl.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const int64_t lanes = pl.lanes[lo];
  const int64_t e = (int64_t)(blockIdx.x - pl.first[lo]) * kCopyThreads + threadIdx.x;
  if (e >= lanes) return;
  uint4* base = pl.base[lo] + e;
  int64_t i0 = 0, i1 = n;
  if (range) {
    i0 = range[1];
    i1 = range[0];
  }
  if (gridDim.y > 1) {
    const int64_t per = (i1 - i0 + gridDim.y - 1) / gridDim.y;
    i0 += per * blockIdx.y;
    i1 = i0 + per < i1 ? i0 + per : i1;
  }
  for (int64_t i = i0; i < i1; i += kMoves) {
    int s[kMoves], d[kMoves];
    uint4 v[kMoves];
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      s[u] = -1;
      d[u] = -1;
      if (i + u < i1) {
        s[u] = src[i + u];
        d[u] = dst ? dst[i + u] : (int)(i + u);
        if ((s[u] >= pl.npages || d[u] >= pl.npages) && status && e == 0) set_status(status, M3_ERR_STATE);
        if (s[u] >= pl.npages || d[u] >= pl.npages || (s[u] < 0 && !zero_neg)) d[u] = -1;
        if (d[u] < 0 || s[u] == d[u]) d[u] = -1;
      }
    }
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      v[u] = make_uint4(0, 0, 0, 0);
      if (d[u] >= 0 && s[u] >= 0) {
        bool fwd = false;
#pragma unroll
        for (int w = 0; w < u; ++w) fwd |= d[w] == s[u];
        if (!fwd) v[u] = __ldcs(base + s[u] * lanes);
      }
    }
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      if (d[u] < 0) continue;
#pragma unroll
      for (int w = 0; w < u; ++w)
        if (s[u] >= 0 && d[w] == s[u]) v[u] = v[w];  // the last such move wins
      base[d[u] * lanes] = v[u];
    }
  }
}

constexpr int kOneCta = 1024;

// Exclusive prefix sum of a flag over the block; *total its sum.  All threads call it.
__device__ __forceinline__ int block_rank(bool flag, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned m = __ballot_sync(0xffffffffu, flag);
  if (lane == 0) warp_sums[warp] = __popc(m);
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kOneCta / 32; ++w) {
    const int c = warp_sums[w];
    if (w < warp) before += c;
    all += c;
  }
  __syncthreads();
  *total = all;
  return before + __popc(m & ((1u << lane) - 1));
}

// Entry i takes the i-th lowest free page; an entry whose source is no live page, and one past the
// last free page, gets -1.
__global__ void __launch_bounds__(kOneCta)
    pages_take_kernel(int npages, int32_t* live, int64_t n, const int32_t* src, int32_t* dst, int* status) {
  __shared__ int sums[kOneCta / 32];
  int64_t taken = 0;
  for (int64_t p0 = 0; p0 < npages && taken < n; p0 += kOneCta) {
    const int64_t p = p0 + threadIdx.x;
    int total;
    const int64_t r = taken + block_rank(p < npages && live[p] == 0, sums, &total);
    if (p < npages && live[p] == 0 && r < n) dst[r] = (int)p;
    taken += total;
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < n; i += kOneCta) {
    const int s = src[i];
    const bool ok = s < 0 || (s < npages && live[s] != 0);
    if (!ok || i >= taken) {
      dst[i] = -1;
      set_status(status, M3_ERR_STATE);
    }
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < n; i += kOneCta)
    if (dst[i] >= 0) live[dst[i]] = 1;
}

__global__ void __launch_bounds__(256) pages_free_kernel(int64_t npages, int32_t* live, int64_t n, const int32_t* idx,
                                                         int* status) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int p = idx[i];
  if (p >= npages) set_status(status, M3_ERR_STATE);
  else if (p >= 0) live[p] = 0;
}

// map[p]: the page's new place (-1: free); order[i]: the page that page i comes from (-1 behind the live
// ones); count[0]: live pages, count[1]: the pages at the front that stay where they are.
__global__ void __launch_bounds__(kOneCta)
    pages_plan_kernel(int npages, int32_t* live, int32_t* map, int32_t* order, int32_t* count) {
  __shared__ int sums[kOneCta / 32];
  int at = 0, stay = npages;
  for (int p0 = 0; p0 < npages; p0 += kOneCta) {
    const int p = p0 + threadIdx.x;
    const bool on = p < npages && live[p] != 0;
    int total;
    const int r = at + block_rank(on, sums, &total);
    if (on) order[r] = p;
    if (p < npages) map[p] = on ? r : -1;
    if (stay == npages && total < (npages - p0 < kOneCta ? npages - p0 : kOneCta)) {
      // the first free page is in this window: the live pages before it stay
      int dummy;
      const int free_rank = block_rank(p < npages && !on, sums, &dummy);
      if (p < npages && !on && free_rank == 0) count[1] = p;
      stay = 0;
    }
    at += total;
  }
  if (stay == npages && threadIdx.x == 0) count[1] = npages;
  if (threadIdx.x == 0) count[0] = at;
  for (int p = threadIdx.x; p < npages; p += kOneCta) {
    if (p >= at) order[p] = -1;
    live[p] = p < at;
  }
}

// The blocks of every buffer; false when they exceed the grid.
bool plan_copy(const m3_pages& pg, CopyPlan* pl, uint32_t* blocks) {
  pl->nbuf = pg.nbuf;
  pl->npages = pg.npages;
  int64_t at = 0;
  for (int j = 0; j < pg.nbuf; ++j) {
    pl->first[j] = (uint32_t)at;
    pl->base[j] = static_cast<uint4*>(pg.base[j]);
    pl->lanes[j] = pg.bytes[j] / 16;
    at += (pl->lanes[j] + kCopyThreads - 1) / kCopyThreads;
    if (at > 0x7fffffff) return false;
  }
  pl->first[pg.nbuf] = (uint32_t)at;
  *blocks = (uint32_t)at;
  return true;
}

cudaError_t launch_copy(const m3_pages& pg, int64_t n, const int32_t* src, const int32_t* dst, const int32_t* range,
                        int zero_neg, unsigned split, int* status, cudaStream_t stream) {
  CopyPlan pl;
  uint32_t blocks = 0;
  if (!plan_copy(pg, &pl, &blocks)) return cudaErrorInvalidConfiguration;
  if (blocks == 0) return cudaSuccess;
  pages_copy_kernel<<<dim3(blocks, split), kCopyThreads, 0, stream>>>(pl, n, src, dst, range, zero_neg, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pages_copy(const m3_pages& pg, int64_t n, const int32_t* src, const int32_t* dst, int* status,
                              cudaStream_t stream) {
  return launch_copy(pg, n, src, dst, nullptr, 0, 1, status, stream);
}

cudaError_t launch_pages_fork(const m3_pages& pg, int32_t* live, int64_t n, const int32_t* src, int32_t* dst,
                              int* status, cudaStream_t stream) {
  pages_take_kernel<<<1, kOneCta, 0, stream>>>(pg.npages, live, n, src, dst, status);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // sources are live, destinations free and distinct: the moves are independent
  const int64_t split = (n + kMoves - 1) / kMoves;
  return launch_copy(pg, n, src, dst, nullptr, 1, (unsigned)(split < 64 ? split : 64), nullptr, stream);
}

cudaError_t launch_pages_free(int64_t npages, int32_t* live, int64_t n, const int32_t* idx, int* status,
                              cudaStream_t stream) {
  const int64_t grid = (n + 255) / 256;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  pages_free_kernel<<<(unsigned)grid, 256, 0, stream>>>(npages, live, n, idx, status);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const m3_pages& pg, int32_t* live, int32_t* map, int32_t* order, int32_t* count,
                                 cudaStream_t stream) {
  pages_plan_kernel<<<1, kOneCta, 0, stream>>>(pg.npages, live, map, order, count);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_copy(pg, 0, order, nullptr, count, 0, 1, nullptr, stream);
}

}  // namespace m3
