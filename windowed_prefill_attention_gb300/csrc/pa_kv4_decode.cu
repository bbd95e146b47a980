// Split-KV flash decode over the paged 4-bit KV pool (sm_103a): one new query
// token per sequence attends to its visible keys (the mask of pa_decode).
//
// Bound by HBM: a key of one kv head is 296 bytes (128 + 16 + 4 for K and for V)
// for 2 x G x 512 flops.  A block is one tile of the pool, 4736 contiguous bytes, so
// one bulk copy brings in its codes and scales, already in an order that 16-byte
// reads take without bank conflicts.
//
// Work split: a (sequence, kv head) pair's visible blocks are cut into runs of
// equal length, as many as make the longest run of the launch short and fill the
// warps that the GPU holds at once.  A warp takes one run and shares nothing: it has a
// ring of tiles and a softmax of its own and writes a partial (row reference, row
// sum, O), or bf16 out where its run is the whole pair; there is no barrier, so no warp
// waits for a slower one.  A second kernel joins a pair's partials in the order of the
// runs (a call's result does not depend on scheduling), spread over the whole GPU.
//
// Products on warp-level MMAs (m16n8k16, fp16 operands, fp32 sums) in the
// transposed orientation, S^T = K Q^T and O^T = V^T P^T: keys and dims fill M, the
// G <= 8 query rows N.  A code times its block scale is exact in fp16, so K and V
// enter exactly; the query enters as fp16 through a power of two per row, exactly
// but for values under 2^-20 of the row's largest.
// V's row scale s enters through the weights, and a row has two references: m follows its scores
// y (log2), n its z = y + d, 2^d the power of two above s.  p = 2^(y - m) goes into the sum of
// weights, P' = p s 2^(m - n) into the product: in fp16's range whatever the scales, and held
// against the row's largest p s, not its largest s: a key of a huge V row and no weight costs
// the others nothing.  P' is rounded to fp16: 2^-11 of each, far under the rounding of the
// bf16 output, and at most 2^-31 of the largest where fp16's normal range ends.
// Scores, references, sums and O are fp32.  A reference moves only when a y or z passes the largest one at its last
// move by 2^8, so the common block needs a vote and no reduction over the warp.
// What is joined is O in units of 2^n, with n and the logarithm of the weights' sum: a mean of values near
// the top of fp32's range never passes through their sum, and a run of small values does not lose its weight.
// Dims are permuted so that a thread's operands are whole words: thread (g, t) of
// a warp reads dims [64 t, 64 t + 64) of keys g and g + 8 for K, dims [32 g, 32 g +
// 32) of keys 2t, 2t + 1, 2t + 8, 2t + 9 for V (whose codes of a key pair are
// interleaved by masks before they are widened, so that a pair of fp16 values is
// one dim of both keys).
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pa_decode.cuh"
#include "pa_internal.h"
#include "pa_kv4.cuh"
#include "pa_ptx.cuh"

namespace pa {
namespace {

// Two tiles a step, whose scores share one vote and whose products are independent
// chains: some 520 instructions a tile with all set-up (70 more one at a time) and as many registers
// as 8 warps an SM leave.  5 contexts of 120 to 200 thousand tokens, 237 MB: 46.9 us (5.0 TB/s; the copies
// alone take 40.6), 64 windowed contexts, 157 MB: 35.9.  With the scales under a normaliser of the
// largest one so far, which lost what lay far below it, 45.7 and 35.7, and then: one tile a
// step on 12 warps 48.4, on 8 warps 51.7, on 16 warps of 128 registers 52.6; three steps in the ring
// 47.6; queries in shared memory 47.0.
constexpr int kWarps = 4;       // a CTA's, which share nothing until its runs are joined
constexpr int kCtasPerSm = 2;
constexpr int kStages = 2;      // steps, of two tiles each, of a warp in flight or in work
constexpr int kStepBytes = 2 * kT4Bytes;
constexpr int kSmBars = kWarps * kStages * kStepBytes;
constexpr int kSmem = kSmBars + kWarps * kStages * 8 + 128;
constexpr float kMargin = 8.f;  // log2: how far y and z may pass the largest ones at their references' last move
constexpr float kLift = 7.f;    // m is that largest y, n that largest z - kLift: p <= 2^8, P' <= 2^15
// (2^(m - n) is at most 2^107: d is at least -99, the append's least scale being 2^-100)
constexpr int kMergeWarps = 32;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
// (not volatile: the compiler may order products freely)
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float lg2f(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A maximum as what exponents are taken from: where there is nothing (or NaN, which stays in the sums) not -inf.
__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float lds_f32(uint32_t addr) { return __uint_as_float(lds32(addr)); }

// Run i of n over a pair's blocks begins at this one: after whole steps of two blocks.
__device__ __forceinline__ int run_start(int i, int n_blocks, int n) {
  return min(n_blocks, 2 * (int)((long long)i * ((n_blocks + 1) / 2) / n));
}

// The pair's query rows as fp16 B fragments of Q^T, each row scaled by the power of two
// that puts its absmax in [64, 128): lane (row, t) holds dims [64 t, 64 t + 64), q[w] those
// at 8 w + {0, 1}, {2, 3} (k-step 2 w) and {4, 5}, {6, 7} (k-step 2 w + 1), as the K
// operand has them.  Rows >= G are zero.
// c: the factors of rows 2 t and 2 t + 1 (2^-k sm_scale log2 e).
__device__ __forceinline__ void load_q(const Kv4DecodeParams& p, const DecSeq& d, int g, int lane, uint4 (&q)[8], float (&c)[2]) {
  const int row = lane >> 2, t = lane & 3;
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  if (row < p.G) {
    const uint4* src = reinterpret_cast<const uint4*>(p.q + ((size_t)d.q_row * p.HQ + (size_t)g * p.G + row) * kHeadDim + 64 * t);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = src[i];  // not through the read-only path: out may be q
  }
  uint32_t am2 = 0u;  // magnitudes of bf16 order as their bits
#pragma unroll
  for (int i = 0; i < 8; ++i)
    am2 = __vmaxu2(am2, __vmaxu2(__vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu),
                                 __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu)));
  uint32_t am = max(am2 & 0xffffu, am2 >> 16);
  am = max(am, __shfl_xor_sync(kAll, am, 1));
  am = max(am, __shfl_xor_sync(kAll, am, 2));
  const int k = am > 0u ? min(126, 133 - (int)(am >> 7)) : 0;  // 2^-k stays a normal number
  const float mul = __uint_as_float((uint32_t)(127 + k) << 23);
  const float mine = row < p.G ? __uint_as_float((uint32_t)(127 - k) << 23) * p.sm_scale_log2 : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = pack_f16x2(__uint_as_float(u[e] << 16) * mul, __uint_as_float(u[e] & 0xffff0000u) * mul);
    q[i] = make_uint4(h[0], h[1], h[2], h[3]);
  }
  c[0] = __shfl_sync(kAll, mine, 8 * t);
  c[1] = __shfl_sync(kAll, mine, 8 * t + 4);
}

// A lane's element k of O: row 2 t + (k >= 8), dims 32 g + 4 (k % 8) .. + 3.
__device__ __forceinline__ float4 o_element(const float (&o)[16][4], int k) {
  const int e = k >> 3, m = 2 * (k & 7);
  return make_float4(o[m][e], o[m][2 + e], o[m + 1][e], o[m + 1][2 + e]);
}

template <class Table>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) kv4_decode_kernel(const __grid_constant__ Kv4DecodeParams p,
                                                                             const __grid_constant__ Table tab) {
  extern __shared__ uint8_t draw[];
  const uint32_t sbase = (smem_u32(draw) + 127u) & ~127u;
  const int HKV = p.HKV;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const WaitCtl wc{p.err, p.wait_ns};
  const uint32_t slot0 = sbase + (uint32_t)(warp * kStages * kStepBytes);
  const uint32_t bar0 = sbase + kSmBars + (uint32_t)(warp * kStages * 8);
  dependents_may_start();  // the merge waits for all of this grid anyway
  const int run = blockIdx.x * kWarps + warp;
  if (run >= p.n_runs) return;
  if (lane < kStages) mbar_init(bar0 + 8 * lane, 1);
  fence_mbar_init();
  __syncwarp();  // the warp's barriers are its own
  // the run's pair: at or behind that of the CTA's first run
  int s = Table::kHints ? tab.cta_seq[blockIdx.x] : 0;
  while (s + 1 < p.n_seq && tab.seq[s + 1].z <= run) ++s;
  const int n_runs = tab.seq[s].w, pair_run = run - tab.seq[s].z, g = pair_run / n_runs;
  const DecSeq d = dec_seq(p, tab, s);
  const int i0 = run_start(pair_run - g * n_runs, d.n_vis, n_runs);
  const int n_mine = run_start(pair_run - g * n_runs + 1, d.n_vis, n_runs) - i0;

  // 1. Tiles: step j is blocks 2 j and 2 j + 1 of the run.  Lane i of a batch holds the
  // addresses of step 32 b + i's (nullptr: behind the run, or a page outside the pool),
  // the next batch's while this one is in work, and issues its copies itself.  Where
  // neither has a tile the slot's phase is completed at once.
  struct Step {
    const uint8_t* tile[2];
  };
  const int n_steps = (n_mine + 1) / 2;
  const int32_t* pages = p.block_table + (size_t)(p.bt_row0 + s) * p.bt_stride;
  wait_for_previous();
  auto look_up = [&](int b) {
    Step r;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 64 * b + 2 * lane + e;
      r.tile[e] = nullptr;
      if (i < n_mine) {
        const int page = __ldcg(pages + dec_block(d, i0 + i));
        if (page < 0 || page >= p.n_pool) record_bad_page(p.err);  // never dereferenced
        else r.tile[e] = p.pool + ((size_t)page * HKV + g) * kT4Bytes;
      }
    }
    return r;
  };
  auto issue = [&](int j, const Step& from, uint32_t slot, uint32_t bar) {
    if (lane == (j & 31)) {
      const uint32_t bytes = (from.tile[0] ? kT4Bytes : 0) + (from.tile[1] ? kT4Bytes : 0);
      if (bytes == 0) {
        mbar_arrive(bar);
      } else {
        mbar_expect_tx(bar, bytes);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (from.tile[e]) bulk_load(slot + e * kT4Bytes, from.tile[e], kT4Bytes, bar);
      }
    }
  };
  Step step = look_up(0);
  int issued = min(kStages, n_steps);
  for (int j = 0; j < issued; ++j) issue(j, step, slot0 + (uint32_t)(j * kStepBytes), bar0 + 8 * j);
  Step next_step = look_up(1);
  uint32_t have0 = __ballot_sync(kAll, step.tile[0] != nullptr), have1 = __ballot_sync(kAll, step.tile[1] != nullptr);

  bool ok = true;  // false once a wait gave up: the warp computes nothing more
  uint4 q[8];
  float c[2];
  load_q(p, d, g, lane, q, c);
  float m_lo = -INFINITY, m_hi = -INFINITY, n_lo = -INFINITY, n_hi = -INFINITY;  // references
  float top_m_lo = -INFINITY, top_m_hi = -INFINITY, top_n_lo = -INFINITY, top_n_hi = -INFINITY;  // what they hold up to
  float r_lo = 0.f, r_hi = 0.f;                                                  // 2^(m - n)
  float l_lo = 0.f, l_hi = 0.f;                                                  // the lane's share of the sums
  // the lane's offsets in a tile
  const int k_at0 = kv4_piece(gq, 2 * tq), k_at1 = kv4_piece(gq, 2 * tq + 1), kb_at = kT4Block + gq * 16 + 4 * tq;
  const int v_at0 = kT4V + kv4_piece(2 * tq, gq), v_at1 = kT4V + kv4_piece(2 * tq + 1, gq), vb_at = kT4Block + 256 + 32 * tq + 2 * gq;
  const int row_at = kT4Row + 4 * gq;
  const int last = d.n_vis - 1 - i0;  // the pair's last block, which may end with keys behind the query
  float o[16][4];
#pragma unroll
  for (int mt = 0; mt < 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

  // 2. The steps, in turn, as their copies land.
  int it = 0;
  uint32_t kb = slot0, bar = bar0, phase = 0u;  // step `it`'s slot
#pragma unroll 1
  for (; it < n_steps; ++it) {
    if (!__all_sync(kAll, mbar_wait(bar, phase, wc, 70))) {
      ok = false;
      break;
    }
    const bool h0 = (have0 >> (it & 31)) & 1u, h1 = (have1 >> (it & 31)) & 1u;
    if (h0 || h1) {
      // S^T = K Q^T: keys gq, gq + 8 of both blocks x rows 2tq, 2tq + 1
      float sacc[2][2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int m = 0; m < 2; ++m) sacc[e][m][0] = sacc[e][m][1] = sacc[e][m][2] = sacc[e][m][3] = 0.f;
      __half2 ks[2][2][4];  // block scales of the thread's four blocks of keys gq and gq + 8, as pairs
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t w = lds32(kb + e * kT4Bytes + kb_at + 128 * r);
          const uint32_t lo = e4m3x2_to_f16(w & 0xffffu), hi = e4m3x2_to_f16(w >> 16);
          const __half2 hl = *reinterpret_cast<const __half2*>(&lo), hh = *reinterpret_cast<const __half2*>(&hi);
          ks[e][r][0] = __low2half2(hl), ks[e][r][1] = __high2half2(hl);
          ks[e][r][2] = __low2half2(hh), ks[e][r][3] = __high2half2(hh);
        }
#pragma unroll
      for (int j = 0; j < 2; ++j) {  // pieces 2tq + j: dims 64 tq + 32 j + [0, 32)
        uint32_t w[2][2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint4 v = lds128(kb + e * kT4Bytes + (j ? k_at1 : k_at0) + 1024 * r);
            w[e][r][0] = v.x, w[e][r][1] = v.y, w[e][r][2] = v.z, w[e][r][3] = v.w;
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 qb = q[4 * j + i];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t a0[4], a1[4];
            e2m1x8_to_f16(w[e][0][i], a0);
            e2m1x8_to_f16(w[e][1][i], a1);
            const uint32_t s0 = *reinterpret_cast<const uint32_t*>(&ks[e][0][2 * j + i / 2]);
            const uint32_t s1 = *reinterpret_cast<const uint32_t*>(&ks[e][1][2 * j + i / 2]);
            const uint32_t x[4] = {mul_f16x2(a0[0], s0), mul_f16x2(a1[0], s1), mul_f16x2(a0[1], s0), mul_f16x2(a1[1], s1)};
            const uint32_t y[4] = {mul_f16x2(a0[2], s0), mul_f16x2(a1[2], s1), mul_f16x2(a0[3], s0), mul_f16x2(a1[3], s1)};
            mma(sacc[e][0], x, qb.x, qb.y);
            mma(sacc[e][1], y, qb.z, qb.w);
          }
        }
      }
      float y[2][4], z[2][4], vs[2][2];  // [e][row of 2][key of 2]; of the keys V's row scales
      uint32_t vbs[2][4];  // V's block scales of keys 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t at = kb + e * kT4Bytes;
        const float ks0 = lds_f32(at + row_at), ks1 = lds_f32(at + row_at + 32);
        float d[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t bits = lds32(at + row_at + 64 + 32 * r);  // not negative
          vs[e][r] = __uint_as_float(bits);
          d[r] = scale_exponent(bits);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x = sacc[e][0][k] + sacc[e][1][k], f = (k < 2 ? ks0 : ks1) * c[k & 1];
          y[e][k] = x * f;
          z[e][k] = fmaf(x, f, d[k >> 1]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) vbs[e][k] = lds16(at + vb_at + 16 * (k & 1) + 128 * (k >> 1));
      }
      if (!(h0 && h1) || 2 * it + 1 >= last) {  // blocks that are not there, keys behind the query: whatever their slots hold
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int n_keys = !(e ? h1 : h0) ? 0 : (2 * it + e == last ? d.t % kPage + 1 : kPage);
          if (gq >= n_keys) y[e][0] = y[e][1] = z[e][0] = z[e][1] = -INFINITY, vs[e][0] = 0.f;
          if (gq + 8 >= n_keys) y[e][2] = y[e][3] = z[e][2] = z[e][3] = -INFINITY, vs[e][1] = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k)  // e4m3 has a NaN (e2m1 has none)
            if (2 * tq + (k & 1) + 8 * (k >> 1) >= n_keys) vbs[e][k] = 0u;
        }
      }
      float bm_lo = fmaxf(fmaxf(y[0][0], y[0][2]), fmaxf(y[1][0], y[1][2])), bm_hi = fmaxf(fmaxf(y[0][1], y[0][3]), fmaxf(y[1][1], y[1][3]));
      float bn_lo = fmaxf(fmaxf(z[0][0], z[0][2]), fmaxf(z[1][0], z[1][2])), bn_hi = fmaxf(fmaxf(z[0][1], z[0][3]), fmaxf(z[1][1], z[1][3]));
      if (__any_sync(kAll, bm_lo > top_m_lo || bm_hi > top_m_hi || bn_lo > top_n_lo || bn_hi > top_n_hi)) {  // new references
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
          bm_lo = fmaxf(bm_lo, __shfl_xor_sync(kAll, bm_lo, sh));
          bm_hi = fmaxf(bm_hi, __shfl_xor_sync(kAll, bm_hi, sh));
          bn_lo = fmaxf(bn_lo, __shfl_xor_sync(kAll, bn_lo, sh));
          bn_hi = fmaxf(bn_hi, __shfl_xor_sync(kAll, bn_hi, sh));
        }
        const float mm_lo = fmaxf(m_lo, bm_lo), mm_hi = fmaxf(m_hi, bm_hi);  // finite: key 0 of a block is visible
        const float nn_lo = fmaxf(n_lo, bn_lo - kLift), nn_hi = fmaxf(n_hi, bn_hi - kLift);
        const float f_lo = ex2f(n_lo - nn_lo), f_hi = ex2f(n_hi - nn_hi);
        l_lo *= ex2f(m_lo - mm_lo);
        l_hi *= ex2f(m_hi - mm_hi);
#pragma unroll
        for (int mt = 0; mt < 16; ++mt) {
          o[mt][0] *= f_lo;
          o[mt][1] *= f_hi;
          o[mt][2] *= f_lo;
          o[mt][3] *= f_hi;
        }
        m_lo = mm_lo, m_hi = mm_hi, n_lo = nn_lo, n_hi = nn_hi;
        top_m_lo = m_lo + kMargin, top_m_hi = m_hi + kMargin, top_n_lo = n_lo + (kLift + kMargin), top_n_hi = n_hi + (kLift + kMargin);
        r_lo = ex2f(m_lo - n_lo), r_hi = ex2f(m_hi - n_hi);
      }
      uint32_t pb[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float p0 = ex2f(y[e][0] - m_lo), p1 = ex2f(y[e][1] - m_hi), p2 = ex2f(y[e][2] - m_lo), p3 = ex2f(y[e][3] - m_hi);
        l_lo += p0 + p2;
        l_hi += p1 + p3;
        // p s first: what the factor 2^(m - n) alone would take out of fp32's range has no weight
        pb[e][0] = transpose8x8(pack_f16x2(p0 * vs[e][0] * r_lo, p1 * vs[e][0] * r_hi));
        pb[e][1] = transpose8x8(pack_f16x2(p2 * vs[e][1] * r_lo, p3 * vs[e][1] * r_hi));
      }
      // O^T += V^T P^T.  Row gq of m-tile mt is dim 32 gq + 2 mt, row gq + 8 dim 32 gq + 2 mt + 1.
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t vs2[2][2];  // block scales of the thread's two blocks: [key pair][block]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t w = __byte_perm(vbs[e][2 * r], vbs[e][2 * r + 1], 0x5140);
          vs2[r][0] = e4m3x2_to_f16(w & 0xffffu);
          vs2[r][1] = e4m3x2_to_f16(w >> 16);
        }
        uint32_t w[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 r = lds128(kb + e * kT4Bytes + ((k & 1) ? v_at1 : v_at0) + 1024 * (k >> 1));
          w[k][0] = r.x, w[k][1] = r.y, w[k][2] = r.z, w[k][3] = r.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // dims 32 gq + 8 i .. + 7: m-tiles 4 i .. 4 i + 3
          uint32_t ev0[4], od0[4], ev8[4], od8[4];
          constexpr uint32_t kLow = 0x0f0f0f0fu;
          e2m1x8_to_f16((w[0][i] & kLow) | ((w[1][i] << 4) & ~kLow), ev0);
          e2m1x8_to_f16(((w[0][i] >> 4) & kLow) | (w[1][i] & ~kLow), od0);
          e2m1x8_to_f16((w[2][i] & kLow) | ((w[3][i] << 4) & ~kLow), ev8);
          e2m1x8_to_f16(((w[2][i] >> 4) & kLow) | (w[3][i] & ~kLow), od8);
          const uint32_t s0 = vs2[0][i / 2], s8 = vs2[1][i / 2];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint32_t a[4] = {mul_f16x2(ev0[b], s0), mul_f16x2(od0[b], s0), mul_f16x2(ev8[b], s8), mul_f16x2(od8[b], s8)};
            mma(o[4 * i + b], a, pb[e][0], pb[e][1]);
          }
        }
      }
    }
    __syncwarp();  // every lane is done with this slot before it is refilled
    const int nx = it + kStages;
    if (nx < n_steps) {
      issue(nx, ((nx ^ it) & 32) ? next_step : step, kb, bar);
      ++issued;
    }
    kb += kStepBytes;
    bar += 8;
    if (bar == bar0 + 8 * kStages) kb = slot0, bar = bar0, phase ^= 1u;
    if ((it & 31) == 31) {
      step = next_step;
      have0 = __ballot_sync(kAll, step.tile[0] != nullptr);
      have1 = __ballot_sync(kAll, step.tile[1] != nullptr);
      next_step = look_up((it >> 5) + 2);
    }
  }
  // after a wait gave up: the copies it did not wait for land before the ring is used again (bounded)
  if (!ok) {
    if (lane == 0)
      for (int i = it; i < issued; ++i)
        (void)mbar_wait_drain(bar0 + 8 * (i % kStages), (uint32_t)(i / kStages) & 1u, kDrainNs);
    __syncwarp();
  }

  // 3. The run's result.
#pragma unroll
  for (int sh = 4; sh < 32; sh <<= 1) {
    l_lo += __shfl_xor_sync(kAll, l_lo, sh);
    l_hi += __shfl_xor_sync(kAll, l_hi, sh);
  }
  if (n_runs == 1) {  // l is 0 where every page was outside the pool
    const float f_lo = l_lo == 0.f ? 0.f : ex2f(n_lo - m_lo) / l_lo, f_hi = l_hi == 0.f ? 0.f : ex2f(n_hi - m_hi) / l_hi;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (2 * tq + e >= p.G) continue;
      uint4* dst = reinterpret_cast<uint4*>(p.out + ((size_t)d.q_row * p.HQ + (size_t)g * p.G + 2 * tq + e) * kHeadDim +
                                            32 * gq);
      const float f = e ? f_hi : f_lo;
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float4 a = o_element(o, 8 * e + k), b = o_element(o, 8 * e + k + 1);
        const __nv_bfloat162 r[4] = {__floats2bfloat162_rn(a.x * f, a.y * f), __floats2bfloat162_rn(a.z * f, a.w * f),
                                     __floats2bfloat162_rn(b.x * f, b.y * f), __floats2bfloat162_rn(b.z * f, b.w * f)};
        const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
        dst[k / 2] = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
    return;
  }
  // The partial.  Where the CTA's runs are all of this pair they are joined first, through
  // the rings: the first run's partial is then the CTA's.
  const int r0 = tab.seq[s].z + g * n_runs, cta0 = blockIdx.x * kWarps;
  const bool joined = cta0 >= r0 && cta0 + kWarps <= r0 + n_runs;
  float4* part = reinterpret_cast<float4*>(p.part) + (size_t)(joined ? cta0 : run) * kKv4Part;
  float2* nw = p.nw + (size_t)(joined ? cta0 : run) * 8;
  const float w_lo = m_lo + lg2f(l_lo), w_hi = m_hi + lg2f(l_hi);  // -inf without a key
  if (!joined) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (2 * tq + (k >> 3) >= p.G) continue;
      part[k * 32 + lane] = o_element(o, k);
    }
    if (gq == 0) {  // rows 2 tq and 2 tq + 1
      nw[2 * tq] = make_float2(n_lo, w_lo);
      nw[2 * tq + 1] = make_float2(n_hi, w_hi);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float4 a = o_element(o, k);
    sts128(slot0 + (uint32_t)(k * 32 + lane) * 16,
           make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(a.z), __float_as_uint(a.w)));
  }
  if (gq == 0) sts128(slot0 + kKv4Part * 16 + 16 * tq, make_uint4(__float_as_uint(n_lo), __float_as_uint(w_lo),
                                                                __float_as_uint(n_hi), __float_as_uint(w_hi)));
  __syncthreads();  // all warps of the CTA come here: the choice is the CTA's
  float f[2][kWarps];  // the warps' factors of rows 2 tq and 2 tq + 1
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t at = sbase + kKv4Part * 16 + 16 * tq + 8 * e;
    float n[kWarps], wt[kWarps], n_max = -INFINITY, w_max = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      n[w] = lds_f32(at + w * kStages * kStepBytes), wt[w] = lds_f32(at + w * kStages * kStepBytes + 4);
      n_max = fmaxf(n_max, n[w]), w_max = fmaxf(w_max, wt[w]);
    }
    const float n_ref = finite_ref(n_max), w_ref = finite_ref(w_max);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      f[e][w] = ex2f(n[w] - n_ref);
      l += ex2f(wt[w] - w_ref);
    }
    if (warp == 0 && gq == 0) nw[2 * tq + e] = make_float2(n_max, w_ref + lg2f(l));
  }
  for (int k = warp; k < 16; k += kWarps) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 v = lds_f32x4(sbase + (uint32_t)(w * kStages * kStepBytes + (k * 32 + lane) * 16));
      const float x = k >= 8 ? f[1][w] : f[0][w];
      a = make_float4(a.x + x * v.x, a.y + x * v.y, a.z + x * v.z, a.w + x * v.w);
    }
    if (2 * tq + (k >> 3) < p.G) part[k * 32 + lane] = a;
  }
}

// The partials of a pair joined.  A warp takes one k (a float4 of every lane) of every
// ways-th partial; a CTA the ways of one or four k of a pair, joined in shared memory
// in a fixed order.
template <class Table>
__global__ void __launch_bounds__(32 * kMergeWarps) kv4_merge_kernel(const __grid_constant__ Kv4DecodeParams p,
                                                                     const __grid_constant__ Table tab, int ways) {
  __shared__ float4 acc_sh[kMergeWarps][32];
  __shared__ float nwl_sh[3][kMergeWarps][32];
  const int s = blockIdx.x / p.HKV, g = blockIdx.x - s * p.HKV;
  const int n_runs = tab.seq[s].w;
  if (n_runs == 1) return;  // the run wrote the pair's output
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, way = warp % ways;
  const int k = blockIdx.y * ((blockDim.x >> 5) / ways) + warp / ways, row = 2 * (lane & 3) + (k >> 3);
  float n = -INFINITY, w = -INFINITY, l = 0.f;  // acc in units of 2^n, the weights' sum l 2^w
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  wait_for_previous();
  dependents_may_start();  // not before: a decode behind this one would hold the registers that this one's CTAs need
  if (row < p.G) {
    // the pair's partials: runs before its first whole CTA, one for each of its whole CTAs, runs behind them
    const int first = tab.seq[s].z + g * n_runs, lead = min(n_runs, (kWarps - first % kWarps) % kWarps);
    const int full = (n_runs - lead) / kWarps, n_parts = n_runs - full * (kWarps - 1);
    const auto part_id = [&](int i) { return (size_t)(first + i + (kWarps - 1) * min(max(i - lead, 0), full)); };
    constexpr int kAtOnce = 8;
    for (int r = way; r < n_parts; r += kAtOnce * ways) {
      float2 nw[kAtOnce];
      float4 v[kAtOnce];
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const bool have = r + e * ways < n_parts;
        const size_t id = part_id(have ? r + e * ways : r);
        nw[e] = __ldcg(p.nw + id * 8 + row);
        v[e] = __ldcg(reinterpret_cast<const float4*>(p.part) + id * kKv4Part + k * 32 + lane);
        if (!have) nw[e] = make_float2(-INFINITY, -INFINITY);
      }
      float n_max = n, w_max = w;
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) n_max = fmaxf(n_max, nw[e].x), w_max = fmaxf(w_max, nw[e].y);
      const float n_ref = finite_ref(n_max), w_ref = finite_ref(w_max);
      const float al = ex2f(n - n_ref);
      l *= ex2f(w - w_ref);
      acc = make_float4(acc.x * al, acc.y * al, acc.z * al, acc.w * al);
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const float f = ex2f(nw[e].x - n_ref);
        l += ex2f(nw[e].y - w_ref);
        acc = make_float4(acc.x + f * v[e].x, acc.y + f * v[e].y, acc.z + f * v[e].z, acc.w + f * v[e].w);
      }
      n = n_max, w = w_max;
    }
  }
  if (ways > 1) {
    acc_sh[warp][lane] = acc;
    nwl_sh[0][warp][lane] = n, nwl_sh[1][warp][lane] = w, nwl_sh[2][warp][lane] = l;
    __syncthreads();
    if (way > 0) return;
    for (int i = 1; i < ways; ++i) n = fmaxf(n, nwl_sh[0][warp + i][lane]), w = fmaxf(w, nwl_sh[1][warp + i][lane]);
    const float n_ref = finite_ref(n), w_ref = finite_ref(w);
    acc = make_float4(0.f, 0.f, 0.f, 0.f), l = 0.f;
    for (int i = 0; i < ways; ++i) {
      const float f = ex2f(nwl_sh[0][warp + i][lane] - n_ref);
      const float4 v = acc_sh[warp + i][lane];
      l += ex2f(nwl_sh[1][warp + i][lane] - w_ref) * nwl_sh[2][warp + i][lane];
      acc = make_float4(acc.x + f * v.x, acc.y + f * v.y, acc.z + f * v.z, acc.w + f * v.w);
    }
  }
  if (row >= p.G) return;
  const float f = l == 0.f ? 0.f : ex2f(n - w) / l;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * f, acc.y * f), hi = __floats2bfloat162_rn(acc.z * f, acc.w * f);
  uint2 out;
  out.x = *reinterpret_cast<const uint32_t*>(&lo);
  out.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(p.out + ((size_t)tab.seq[s].x * p.HQ + (size_t)g * p.G + row) * kHeadDim + 32 * (lane >> 2) + 4 * (k & 7)) = out;
}

}  // namespace

int kv4_decode_warps(int n_sm) { return n_sm * kCtasPerSm * kWarps; }
int kv4_decode_cta_warps() { return kWarps; }

namespace {
template <class Table>
cudaError_t launch(const Kv4DecodeParams& p, const Table& seqs, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kv4_decode_kernel<Table>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = launch_early(kv4_decode_kernel<Table>, dim3((p.n_runs + kWarps - 1) / kWarps), kWarps * 32, kSmem, st, p, seqs);
  if (e != cudaSuccess || p.most_runs < 2) return e;
  const int pairs = p.n_seq * p.HKV, ks = pairs < 64 ? 1 : 4;
  const int most_parts = p.most_runs < kWarps ? p.most_runs : p.most_runs / kWarps + 2 * (kWarps - 1);
  const int ways = std::min(kMergeWarps / ks, (most_parts + 7) / 8);
  return launch_early(kv4_merge_kernel<Table>, dim3((unsigned)pairs, 16 / ks), (unsigned)(32 * ks * ways), 0, st, p, seqs, ways);
}
}  // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeParams& p, const Kv4DecodeSeqs& seqs, cudaStream_t st) {
  if (p.n_seq > kKv4FewSeqs) return launch(p, seqs, st);
  Kv4DecodeTable<kKv4FewSeqs, 1> few;
  for (int i = 0; i < p.n_seq; ++i) few.seq[i] = seqs.seq[i];
  return launch(p, few, st);
}

}  // namespace pa
