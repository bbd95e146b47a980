// Device helpers of the decode kernels (pa_decode.cu, pa_kv4_decode.cu): the
// warp-level products, and a sequence's visible blocks.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "pa_internal.h"

namespace pa {

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8x8 b16 matrix held one row pair per thread (row lane/4, columns 2(lane%4),
// +1) -> its transpose in the same layout.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
// 16-byte chunk c (0..7) of row r of a 128-byte-swizzled box: chunks are
// permuted by the row index mod 8, as the TMA copy writes them.
__device__ __forceinline__ uint32_t swz128(uint32_t half_base, int r, int c) {
  return half_base + (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
}

// A sequence's decode geometry (from the launch's table entry {row, context, earlier blocks}).
struct DecSeq {
  int q_row;   // row of the query token in q / out
  int t;       // its position in the context (n_ctx - 1)
  int vstart;  // visible blocks of the launch's earlier sequences (per kv head)
  int n_sink;  // sink blocks listed ahead of the window run
  int lo;      // first block of the window run (0 with the window off)
  int n_vis;   // visible blocks
};
template <class P, class T>
__device__ __forceinline__ DecSeq dec_seq(const P& p, const T& tab, int s) {
  const int4 e = tab.seq[s];
  DecSeq d;
  d.q_row = e.x;
  d.t = e.y - 1;
  d.vstart = e.z;
  const int last = d.t / kPage;
  d.lo = p.W > 0 ? max(0, last + 1 - p.W) : 0;
  d.n_sink = p.W > 0 ? min(max(p.S, 0), d.lo) : 0;
  d.n_vis = d.n_sink + (last - d.lo + 1);
  return d;
}
// Logical key block of the b-th visible block of a sequence.
__device__ __forceinline__ int dec_block(const DecSeq& d, int b) { return b < d.n_sink ? b : d.lo + (b - d.n_sink); }

}  // namespace pa
