// Page operators (sm_103a): forks of sequences and compaction of the pools.
//
// Fork: row dst of the block table becomes row src's first ceil(n / 16) entries,
// its pages shared; the page of a part-filled last block is copied to a page of
// its own, in every pool, since both sequences will write to it.
//
// Compaction: the pages in use are those that some sequence's next tokens can still
// see.  With L of them, page p < L stays and the r-th page in use from L on moves to
// the r-th unused page below L: the fewest moves, and no move reads a page that
// another writes.
//
// Bound by memory (a page is read once and written once in each pool) and, for a
// few pages, by launches and the chain table entry -> page.  A warp copies 4 KB at
// a time with all its loads in flight before the first store.  200 forks in 24 pools of
// 4-bit tiles, 85 MB: 12.3 us (6.9 TB/s); 3686 moves in 8 pools, 559 MB: 98 us (5.7 TB/s, 6 us
// of it marks and ranks); one fork or a few 2.1 us, a small compaction 6.7 us.
#include <cstdint>
#include <cuda_runtime.h>

#include "pa_early.cuh"
#include "pa_pages.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;
constexpr int kChunk = 4096;  // bytes of a page that a warp copies at a time
constexpr int kPlanThreads = 1024;
constexpr unsigned kAll = 0xffffffffu;

// Bytes [off, off + kChunk) of page `from`, as far as the page goes, to page `to`.
__device__ __forceinline__ void copy_chunk(const pa_part& part, int from, int to, long long off, int lane) {
  const uint8_t* src = static_cast<const uint8_t*>(part.data) + (size_t)from * part.page_bytes + off;
  uint8_t* dst = static_cast<uint8_t*>(part.data) + (size_t)to * part.page_bytes + off;
  const int bytes = (int)min((long long)kChunk, part.page_bytes - off);
  if (((reinterpret_cast<uintptr_t>(part.data) | (uintptr_t)part.page_bytes) & 15) == 0) {
    uint4 v[kChunk / 512];
#pragma unroll
    for (int k = 0; k < kChunk / 512; ++k)
      if (k * 512 + lane * 16 < bytes) v[k] = __ldcs(reinterpret_cast<const uint4*>(src) + k * 32 + lane);
#pragma unroll
    for (int k = 0; k < kChunk / 512; ++k)
      if (k * 512 + lane * 16 < bytes) reinterpret_cast<uint4*>(dst)[k * 32 + lane] = v[k];
  } else {  // pages of whole words only
    for (int k = lane; k < bytes / 4; k += 32) reinterpret_cast<uint32_t*>(dst)[k] = reinterpret_cast<const uint32_t*>(src)[k];
  }
}

// blockIdx.y < n: pool y, a warp a chunk of a fork's part-filled page.  blockIdx.y == n: the table's rows.
template <int kForks, int kParts>
__global__ void __launch_bounds__(kWarps * 32) fork_kernel(const __grid_constant__ ForkParams p,
                                                           const __grid_constant__ ForksN<kForks> forks,
                                                           const __grid_constant__ PagePartsN<kParts> parts) {
  const int warp = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31, n_warps = gridDim.x * kWarps;
  dependents_may_start();
  wait_for_previous();
  if ((int)blockIdx.y == parts.n) {
    for (int f = warp; f < p.n_fork; f += n_warps) {
      const int4 k = forks.fork[f];
      const int32_t* src = p.table + (size_t)k.x * p.stride;
      int32_t* dst = p.table + (size_t)k.y * p.stride;
      if (parts.n == 0 && k.z % kPage != 0 && lane == 0) {  // else the copies report it
        const int from = src[k.z / kPage];
        if (from < 0 || from >= p.n_pool) record_bad_page(p.err);
      }
      for (int i = lane; i < (k.z + kPage - 1) / kPage; i += 32) dst[i] = i < k.z / kPage ? src[i] : k.w;
    }
    return;
  }
  const pa_part part = parts.part[blockIdx.y];
  const int n_chunk = (int)((part.page_bytes + kChunk - 1) / kChunk);
  const long long items = (long long)p.n_fork * n_chunk;
  for (long long i = warp; i < items; i += n_warps) {
    const int f = (int)(i / n_chunk);
    const int4 k = forks.fork[f];
    if (k.z % kPage == 0) continue;  // no part-filled page
    const int from = p.table[(size_t)k.x * p.stride + k.z / kPage];
    if (from < 0 || from >= p.n_pool) {  // never dereferenced
      if (lane == 0) record_bad_page(p.err);
      continue;
    }
    copy_chunk(part, from, k.w, (i - (long long)f * n_chunk) * kChunk, lane);
  }
}

// Entry b of sequence s: whether the sequence has such a block, and whether a token after its last one can see it.
__device__ __forceinline__ bool has_block(int n_ctx, int b) { return b < (n_ctx + kPage - 1) / kPage; }
__device__ __forceinline__ bool in_use(const CompactParams& p, int n_ctx, int b) {
  return p.W <= 0 || b < p.S || b >= n_ctx / kPage + 1 - p.W;
}

template <int kSeqs>
__global__ void __launch_bounds__(256) mark_kernel(const __grid_constant__ CompactParams p,
                                                   const __grid_constant__ ContextsN<kSeqs> ctx) {
  const int s = blockIdx.y, n_ctx = ctx.n_ctx[s];
  for (int b = blockIdx.x * 256 + threadIdx.x; b < p.stride && has_block(n_ctx, b); b += gridDim.x * 256) {
    if (!in_use(p, n_ctx, b)) continue;
    const int page = p.table[(size_t)(p.row0 + s) * p.stride + b];
    if (page < 0 || page >= p.n_pool) record_bad_page(p.err);
    else atomicOr(p.live + (page >> 5), 1u << (page & 31));
  }
}

// Sum of a value over the block's threads before this one, and over all.
__device__ __forceinline__ unsigned long long scan(unsigned long long v, unsigned long long* sums, unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(kAll, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();  // sums is free
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  unsigned long long all = sums[lane];  // every warp scans the warps' sums: 32 of them
  static_assert(kPlanThreads == 32 * 32, "a sum for each lane");
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(kAll, all, o);
    if (lane >= o) all += u;
  }
  total = __shfl_sync(kAll, all, 31);
  const unsigned long long before = warp > 0 ? __shfl_sync(kAll, all, warp - 1) : 0ull;
  return before + inc - v;
}

// One CTA: counts the pages in use, pairs movers and holes by rank.
__device__ __forceinline__ void plan_moves(const CompactParams& p, const uint32_t* live_bits) {
  __shared__ unsigned long long sums[kPlanThreads / 32];
  const int n_words = (p.n_pool + 31) / 32, per = (n_words + kPlanThreads - 1) / kPlanThreads;
  const int w0 = min(n_words, (int)threadIdx.x * per), w1 = min(n_words, w0 + per);
  unsigned long long mine = 0, total, moves;
  for (int w = w0; w < w1; ++w) mine += __popc(live_bits[w]);
  (void)scan(mine, sums, total);
  const int L = (int)total;
  // bits of word w below page L
  auto below = [&](int w) { return 32 * w + 32 <= L ? kAll : (32 * w >= L ? 0u : (1u << (L - 32 * w)) - 1u); };
  mine = 0;  // holes in the low half, movers in the high one
  for (int w = w0; w < w1; ++w) {
    const uint32_t live = live_bits[w], lo = below(w);
    mine += __popc(~live & lo) + ((unsigned long long)__popc(live & ~lo) << 32);
  }
  const unsigned long long at = scan(mine, sums, moves);
  int hole = (int)(at & kAll), mover = (int)(at >> 32);
  for (int w = w0; w < w1; ++w) {
    const uint32_t live = live_bits[w], lo = below(w);
    for (uint32_t m = ~live & lo; m; m &= m - 1) p.moves[hole++].to = 32 * w + __ffs(m) - 1;
    for (uint32_t m = live & ~lo; m; m &= m - 1) p.moves[mover++].from = 32 * w + __ffs(m) - 1;
  }
  __syncthreads();
  const int n_moves = (int)(moves >> 32);
  for (int r = threadIdx.x; r < n_moves; r += kPlanThreads) p.moved_to[p.moves[r].from] = p.moves[r].to;
  if (threadIdx.x == 0) {
    p.count[0] = L;
    p.count[1] = n_moves;
    *p.n_live = L;
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ CompactParams p) {
  dependents_may_start();
  wait_for_previous();
  plan_moves(p, p.live);
}

// The marks too, in shared memory: a warp a sequence, its entries in use.  (Marks in a launch
// of their own onto cleared words, then the plan: 12.6 us for five sequences, 7.9 so.)
template <int kSeqs>
__global__ void __launch_bounds__(kPlanThreads) mark_plan_kernel(const __grid_constant__ CompactParams p,
                                                                 const __grid_constant__ ContextsN<kSeqs> ctx) {
  extern __shared__ uint32_t live[];
  dependents_may_start();
  for (int w = threadIdx.x; w < (p.n_pool + 31) / 32; w += kPlanThreads) live[w] = 0u;
  wait_for_previous();
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int s = threadIdx.x >> 5; s < p.n_seq; s += kPlanThreads / 32) {
    const int n = (ctx.n_ctx[s] + kPage - 1) / kPage;
    const int lo = p.W > 0 ? min(n, max(0, ctx.n_ctx[s] / kPage + 1 - p.W)) : 0, sink = min(p.S, lo);
    const int32_t* row = p.table + (size_t)(p.row0 + s) * p.stride;
    for (int i = lane; i < sink + n - lo; i += 4 * 32) {
      int page[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = i + 32 * e;
        page[e] = k < sink + n - lo ? row[k < sink ? k : lo + k - sink] : 0;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (i + 32 * e >= sink + n - lo) continue;
        if (page[e] < 0 || page[e] >= p.n_pool) record_bad_page(p.err);
        else atomicOr(live + (page[e] >> 5), 1u << (page[e] & 31));
      }
    }
  }
  __syncthreads();
  plan_moves(p, live);
}

// blockIdx.y < n: the moves in pool y.  blockIdx.y == n: this launch's rows of the new table.
template <int kSeqs, int kParts>
__global__ void __launch_bounds__(kWarps * 32) apply_kernel(const __grid_constant__ CompactParams p,
                                                            const __grid_constant__ ContextsN<kSeqs> ctx,
                                                            const __grid_constant__ PagePartsN<kParts> parts) {
  dependents_may_start();
  wait_for_previous();
  if ((int)blockIdx.y == parts.n) {
    const int L = p.count[0];
    const long long n = (long long)p.n_seq * p.stride, step = (long long)gridDim.x * (kWarps * 32);
    for (long long i = (long long)blockIdx.x * (kWarps * 32) + threadIdx.x; i < n; i += step) {
      const int s = (int)(i / p.stride), b = (int)(i - (long long)s * p.stride);
      const size_t at = (size_t)p.row0 * p.stride + i;
      int32_t e = p.table[at];
      if (has_block(ctx.n_ctx[s], b)) {
        if (!in_use(p, ctx.n_ctx[s], b)) e = -1;
        else if (e >= L && e < p.n_pool) e = p.moved_to[e];
      }
      p.new_table[at] = e;
    }
    return;
  }
  const pa_part part = parts.part[blockIdx.y];
  const int n_chunk = (int)((part.page_bytes + kChunk - 1) / kChunk), lane = threadIdx.x & 31;
  const long long items = (long long)p.count[1] * n_chunk;
  for (long long i = blockIdx.x * kWarps + (threadIdx.x >> 5); i < items; i += gridDim.x * kWarps) {
    const int r = (int)(i / n_chunk);
    const PageMove m = p.moves[r];
    copy_chunk(part, m.from, m.to, (i - (long long)r * n_chunk) * kChunk, lane);
  }
}

// CTAs a pool so that all pools' fill the GPU once, at most one a warp's item.
unsigned columns(long long most_items, int n_parts, int n_sm) {
  const long long want = (most_items + kWarps - 1) / kWarps, fill = (8ll * n_sm + n_parts) / (n_parts + 1);
  const long long n = want < fill ? want : fill;
  return (unsigned)(n < 1 ? 1 : n);
}
long long most_chunks(const PageParts& parts) {
  long long n = 1;
  for (int i = 0; i < parts.n; ++i) n = parts.part[i].page_bytes > n * kChunk ? (parts.part[i].page_bytes + kChunk - 1) / kChunk : n;
  return n;
}

// f with the smaller table where its first n entries fit it.
template <typename F>
void with_few(const PageParts& t, F f) {
  if (t.n > kFewParts) return f(t);
  PagePartsN<kFewParts> few;
  few.n = t.n;
  for (int i = 0; i < t.n; ++i) few.part[i] = t.part[i];
  f(few);
}
template <typename F>
void with_few(const Forks& t, int n, F f) {
  if (n > kFewRows) return f(t);
  ForksN<kFewRows> few;
  for (int i = 0; i < n; ++i) few.fork[i] = t.fork[i];
  f(few);
}
template <typename F>
void with_few(const Contexts& t, int n, F f) {
  if (n > kFewRows) return f(t);
  ContextsN<kFewRows> few;
  for (int i = 0; i < n; ++i) few.n_ctx[i] = t.n_ctx[i];
  f(few);
}

}  // namespace

cudaError_t launch_pages_fork(const ForkParams& p, const Forks& forks, const PageParts& parts, int n_sm, cudaStream_t st) {
  const dim3 grid(columns(p.n_fork * most_chunks(parts), parts.n, n_sm), parts.n + 1);
  cudaError_t e = cudaSuccess;
  with_few(forks, p.n_fork, [&](const auto& f) {
    with_few(parts, [&](const auto& a) {
      e = launch_early(fork_kernel<sizeof(f.fork) / sizeof(int4), sizeof(a.part) / sizeof(pa_part)>, grid, kWarps * 32, 0, st, p, f, a);
    });
  });
  return e;
}

cudaError_t launch_pages_mark(const CompactParams& p, const Contexts& ctx, cudaStream_t st) {
  int most = 1;
  for (int s = 0; s < p.n_seq; ++s) most = imax(most, (ctx.n_ctx[s] + kPage - 1) / kPage);
  with_few(ctx, p.n_seq, [&](const auto& c) { mark_kernel<<<dim3((most + 255) / 256, p.n_seq), 256, 0, st>>>(p, c); });
  return cudaGetLastError();
}

cudaError_t launch_pages_plan(const CompactParams& p, cudaStream_t st) {
  return launch_early(plan_kernel, dim3(1), kPlanThreads, 0, st, p);
}

cudaError_t launch_pages_mark_plan(const CompactParams& p, const Contexts& ctx, cudaStream_t st) {
  const int bytes = (p.n_pool + 31) / 32 * (int)sizeof(uint32_t);
  cudaError_t e = cudaSuccess;
  with_few(ctx, p.n_seq, [&](const auto& c) {
    auto* kernel = mark_plan_kernel<sizeof(c.n_ctx) / sizeof(int)>;
    // the limit is the function's, not this call's: the same from every thread and handle
    if (bytes > 40 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOneCtaPages / 8);
    if (e == cudaSuccess) e = launch_early(kernel, dim3(1), kPlanThreads, (size_t)bytes, st, p, c);
  });
  return e;
}

cudaError_t launch_pages_apply(const CompactParams& p, const Contexts& ctx, const PageParts& parts, int n_sm, cudaStream_t st) {
  const dim3 grid(columns((long long)p.n_pool * most_chunks(parts), parts.n, n_sm), parts.n + 1);
  cudaError_t e = cudaSuccess;
  with_few(ctx, p.n_seq, [&](const auto& c) {
    with_few(parts, [&](const auto& a) {
      e = launch_early(apply_kernel<sizeof(c.n_ctx) / sizeof(int), sizeof(a.part) / sizeof(pa_part)>, grid, kWarps * 32, 0, st, p, c, a);
    });
  });
  return e;
}

}  // namespace pa
