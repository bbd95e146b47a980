// Norm, rotation and append (sm_103a): the step from a layer's projected
// query, key and value rows to what the attention reads.
//
// Per (token, head) row x of 256 values, in fp32 with one rounding at the end:
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r (offset + w)
//   pair i of the rotated dims, turned by a = pos[axis(i)] inv_freq[i]:
//   (y1, y2) -> (y1 cos a - y2 sin a, y2 cos a + y1 sin a)
// so out_e = r (x_e A_e + x_p B_e) with A = (offset + w_e) cos a and B =
// -+(offset + w_p) sin a: A and B depend on the token and not on the head, and
// a warp that takes a token's rows one after another computes them once.
//
// The angle: a position times a frequency in fp32 would be off by 2^-24 of
// the angle (0.01 rad at 10^5 rad).  The frequency is held in turns as a
// 64-bit binary fraction F instead, rounded to the nearest from the double;
// position * F mod 2^64 is the fraction of a turn, in one integer product, off
// by 2^-65 a position (2^-34 of a turn at position 2^31), and the sine and cosine
// are taken of that fraction (|x| <= 1 half turn, error 2^-25 of one).
//
// Bound by memory: 512 bytes read and 512 written per query row (K and V rows
// of the append: 512 read, 260 written).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "pa_qkv.h"

namespace pa {
namespace {

// 20 warps an SM at 96 registers, each with the next four rows (2 KB) on their way
// beside the four in work.  32768 tokens of 18 rows: 104 us, 5.8 TB/s read and
// written; 16 warps 106, 24 (which spill in earnest: here only the appends of half
// pairing do, 32 bytes) 114; without the copies ahead 110; three batches ahead 109.
constexpr int kQkvWarps = 10;
constexpr int kQkvPerSm = 2;  // CTAs
constexpr int kMaxPairs = kHeadDim / 2;
constexpr unsigned kAll = 0xffffffffu;
enum : int { TURN_NONE, TURN_HALVES, TURN_ADJACENT };

// A lane holds dims [8 lane, 8 lane + 8) of a row, as four pairs.
struct Vals {
  float2 v[4];
};
__device__ __forceinline__ Vals unpack8(const uint4 w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  Vals x;
#pragma unroll
  for (int j = 0; j < 4; ++j) x.v[j] = make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
  return x;
}
__device__ __forceinline__ uint4 pack8(const Vals& x) {
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __float22bfloat162_rn(x.v[j]);
    u[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// One value of each of N rows a lane, reduced over the warp's lanes.  Rows are
// halved among the lanes as the distance halves (4 rows: 2 + 1 + 3 shuffles, and
// one each to bring the results back to all lanes, in place of 5 each).
template <bool kMax>
__device__ __forceinline__ float combine(float a, float b) {
  return kMax ? fmaxf(a, b) : a + b;
}
template <int N, bool kMax>
__device__ __forceinline__ void warp_reduce(float (&v)[N], int lane) {
  static_assert(N == 1 || N == 2 || N == 4, "rows of a batch");
  if (N == 4) {
    const bool up = lane & 16;
    const float s0 = up ? v[0] : v[2 % N], s1 = up ? v[1 % N] : v[3 % N];
    const float k0 = up ? v[2 % N] : v[0], k1 = up ? v[3 % N] : v[1 % N];
    v[0] = combine<kMax>(k0, __shfl_xor_sync(kAll, s0, 16));
    v[1 % N] = combine<kMax>(k1, __shfl_xor_sync(kAll, s1, 16));
  }
  if (N >= 2) {
    const int d = N == 4 ? 8 : 16;
    const bool up = lane & d;
    const float s = up ? v[0] : v[1 % N], k = up ? v[1 % N] : v[0];
    v[0] = combine<kMax>(k, __shfl_xor_sync(kAll, s, d));
  }
#pragma unroll
  for (int o = N == 4 ? 4 : (N == 2 ? 8 : 16); o > 0; o >>= 1) v[0] = combine<kMax>(v[0], __shfl_xor_sync(kAll, v[0], o));
  if (N > 1) {
    const float mine = v[0];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(kAll, mine, N == 4 ? 8 * i : 16 * i);
  }
}

// Where a lane's rotation partners are.  Halves: dim i < R/2 pairs with i + R/2,
// a whole lane R/16 lanes away (R is a multiple of 16).  Neighbours: dims 2i and
// 2i + 1, the two of a pair.
template <int kTurn>
__device__ __forceinline__ Vals partners(const uint4 raw, const Vals& x, int from) {
  Vals p;
  if (kTurn == TURN_HALVES) {
    p = unpack8(make_uint4(__shfl_sync(kAll, raw.x, from), __shfl_sync(kAll, raw.y, from), __shfl_sync(kAll, raw.z, from),
                           __shfl_sync(kAll, raw.w, from)));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) p.v[j] = make_float2(x.v[j].y, x.v[j].x);
  }
  return p;
}

// A and B of the lane's eight dims for one set of gains.
struct Turn {
  float2 a[4], b[4];
};
template <int kTurn>
__device__ __forceinline__ void make_turn(const QkvParams& p, const __nv_bfloat16* w, const float2* cs, int lane, int from,
                                          Turn& t) {
  Vals g, gp;
  if (w) {
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(w) + lane);
    g = unpack8(raw);
    if (kTurn != TURN_NONE) gp = partners<kTurn>(raw, g, from);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      g.v[j] = add2(g.v[j], make_float2(p.w_off, p.w_off));
      if (kTurn != TURN_NONE) gp.v[j] = add2(gp.v[j], make_float2(p.w_off, p.w_off));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) g.v[j] = gp.v[j] = make_float2(1.f, 1.f);
  }
  const int d0 = 8 * lane, R = p.rope.rot_dim;
#pragma unroll
  for (int j = 0; j < 4; ++j) t.a[j] = g.v[j], t.b[j] = make_float2(0.f, 0.f);
  if (kTurn != TURN_NONE && d0 < R) {
    const int half = R / 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kTurn == TURN_HALVES) {
        const bool first = d0 < half;
        const float2 c0 = cs[(first ? d0 : d0 - half) + 2 * j], c1 = cs[(first ? d0 : d0 - half) + 2 * j + 1];
        t.a[j] = mul2(g.v[j], make_float2(c0.x, c1.x));
        t.b[j] = mul2(gp.v[j], first ? make_float2(-c0.y, -c1.y) : make_float2(c0.y, c1.y));
      } else {
        const float2 c = cs[(d0 >> 1) + j];
        t.a[j] = mul2(g.v[j], make_float2(c.x, c.x));
        t.b[j] = mul2(gp.v[j], make_float2(-c.y, c.y));
      }
    }
  }
}

// N rows into the pool: scale = absmax / 127, codes rint(x / scale) half to
// even, decided on the IEEE quotients as kv_append_kernel decides them.  Both
// divisions by Markstein's correction of an approximate quotient: with r near
// 1/b, q0 = RN(a r), the remainder a - q0 b is exact in one FMA and q1 = RN(q0 +
// remainder r).  For the scale r = RN(1/127), and q1 = RN(a / 127) for every fp32
// a.  For the codes r is the hardware reciprocal after one Newton step, within
// half a place of 1/b and a little more.  q1 is then off by under 2^-23 of its last
// place before its rounding, and the pairs (a, b) whose quotient comes that near to
// the border of a tie's neighbourhood are few enough to be listed: all round to the
// code that RN(a / b) rounds to, whatever approximation within an ulp the step began
// with, but one: where b's significand is all ones and the step ends below 1/b,
// a = 2^k would get 0 and not 1.  GB300's reciprocal leads the step above it (both
// are held by tests).  Adding 1.5 * 2^23 rounds a quotient
// to an integer, half to even, and leaves the code in the sum's low byte.  A row
// whose remainders could be subnormal is raised by 2^64 first, its scale too.
template <int N>
__device__ __forceinline__ void store_codes(Vals (&x)[N], int lane, int8_t* codes, float* scale_out) {
  float am[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    am[i] = fabsf(x[i].v[0].x);
#pragma unroll
    for (int j = 0; j < 4; ++j) am[i] = max3(am[i], fabsf(x[i].v[j].x), fabsf(x[i].v[j].y));
  }
  warp_reduce<N, true>(am, lane);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    constexpr float kInv127 = 1.0f / 127.0f;
    const float q0 = __fmul_rn(am[i], kInv127);
    const float scale = __fmaf_rn(__fmaf_rn(-q0, 127.f, am[i]), kInv127, q0);
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23
    float b = scale;
    if (scale < 8.077935669463161e-28f) {  // 2^-90
      b *= 18446744073709551616.f;         // 2^64
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i].v[j] = mul2(x[i].v[j], make_float2(18446744073709551616.f, 18446744073709551616.f));
    }
    float r = 0.f;
    if (b > 0.f) {
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b));
      r = __fmaf_rn(r, __fmaf_rn(-r, b, 1.f), r);
    }
    uint32_t f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 q = mul2(x[i].v[j], make_float2(r, r));
      const float2 s = add2(fma2(fma2(q, make_float2(-b, -b), x[i].v[j]), make_float2(r, r), q), make_float2(kRound, kRound));
      f[2 * j] = __float_as_uint(s.x);
      f[2 * j + 1] = __float_as_uint(s.y);
    }
    const uint32_t lo = __byte_perm(__byte_perm(f[0], f[1], 0x0040), __byte_perm(f[2], f[3], 0x0040), 0x5410);
    const uint32_t hi = __byte_perm(__byte_perm(f[4], f[5], 0x0040), __byte_perm(f[6], f[7], 0x0040), 0x5410);
    reinterpret_cast<uint2*>(codes + i * kHeadDim)[lane] = make_uint2(lo, hi);
    if (lane == 0) scale_out[i] = scale;
  }
}

// A warp's rows on their way in: batches of up to four rows of one kind, copied
// asynchronously into two slots of its own, a batch ahead of the one in work, from
// item to item.  A lane reads only bytes that it copied itself.
struct Feed {
  uint32_t at;    // the lane's 16 bytes of slot 0's first row
  int n_fetched;  // batches so far
  int row, r, r1;  // the token's row; its rows r .. r1 are still to come
  int next_row, next_r0, next_r1;  // then those of the next item; row -1: none

  __device__ __forceinline__ void fetch(const QkvParams& p, int lane) {
    if (r >= r1) {
      r = next_r0, r1 = next_r1, row = next_row;
      next_row = -1;
      if (row < 0) r = r1 = 0;
    }
    if (r < r1) {
      const int nk = p.n_q + p.n_k;
      const RowsIn& in = r < p.n_q ? p.q : (r < nk ? p.k : p.v);
      const int first = r < p.n_q ? 0 : (r < nk ? p.n_q : nk), end = r < p.n_q ? p.n_q : (r < nk ? nk : r1);
      const int n = min(min(end, r1) - r, 4);
      const __nv_bfloat16* src = in.p + (size_t)row * in.ts + (size_t)(r - first) * in.hs + 8 * lane;
      const uint32_t dst = at + (n_fetched & 1) * (4 * 512);
      for (int i = 0; i < n; ++i, src += in.hs)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512 * i), "l"(src) : "memory");
      r += n;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++n_fetched;
  }
  // The slot of the batch before the last one fetched, which has landed.
  __device__ __forceinline__ uint32_t slot() const {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    return at + (n_fetched & 1) * (4 * 512);
  }
};

// A row whose mean square (with eps) is below this is raised by 2^76, exactly, and
// eps by its square: the squares of values under 2^-63 leave fp32's normal range.
// Above it what they lose is nothing to the sum; raised, the sum of squares is under
// 2^120 and the smallest nonzero square 2^-114.
constexpr float kTinyMeanSquare = 9.094947017729282e-13f;  // 2^-40
constexpr float kRaise = 75557863725914323419136.f;        // 2^76
// (The test costs 0.1 us of 3.0 for one token, 0.3 of 31.9 and 0.4 of 41.1 for the
// appends, nothing that shows for 32768 tokens; done in place within the batch it
// spilled 184 bytes, and stores held back instead of an early return took 105.5 us.)

__device__ __forceinline__ void raise_row(uint32_t at) {
  uint4 w;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at));
  Vals x = unpack8(w);
#pragma unroll
  for (int j = 0; j < 4; ++j) x.v[j] = mul2(x.v[j], make_float2(kRaise, kRaise));
  w = pack8(x);
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
}

// N rows from their slot, normed and turned (kNorm), stored as bf16 (kCodes
// false; dst: the lane's 16 bytes of the first row) or as codes.  Rows of which
// one's mean square is below `least_ok` are left alone (false).
template <int N, int kTurn, bool kNorm, bool kCodes>
__device__ __forceinline__ bool do_rows(uint32_t src, const Turn& t, int from, float eps, float least_ok, int lane,
                                        uint4* dst, int8_t* codes, float* scales, bool store) {
  uint4 raw[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(raw[i].x), "=r"(raw[i].y), "=r"(raw[i].z), "=r"(raw[i].w)
                 : "r"(src + 512 * i));
  Vals y[N];
  if (kNorm) {
    float ss[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      y[i] = unpack8(raw[i]);
      float2 s = mul2(y[i].v[0], y[i].v[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) s = fma2(y[i].v[j], y[i].v[j], s);
      ss[i] = s.x + s.y;
    }
    warp_reduce<N, false>(ss, lane);
    float least = INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      ss[i] = fmaf(ss[i], 1.f / kHeadDim, eps);
      least = fminf(least, ss[i]);
    }
    if (least < least_ok) return false;  // the same in all lanes
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float r = ss[i] > 0.f ? rsqrtf(ss[i]) : 0.f;  // an all-zero row with eps 0 stays zero
      Vals xp;
      if (kTurn != TURN_NONE) xp = partners<kTurn>(raw[i], y[i], from);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 v = mul2(y[i].v[j], t.a[j]);
        if (kTurn != TURN_NONE) v = fma2(xp.v[j], t.b[j], v);
        y[i].v[j] = mul2(v, make_float2(r, r));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = unpack8(raw[i]);
  }
  if (kCodes) {
    if (store) store_codes<N>(y, lane, codes, scales);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) dst[i * (kHeadDim / 8)] = pack8(y[i]);
  }
  return true;
}

template <int N>
struct Rows {
  static constexpr int value = N;
};

// `n` heads from head `a` of one kind of row of a token, the next batches of the feed.
template <int kTurn, bool kNorm, bool kCodes>
__device__ __forceinline__ void do_heads(const QkvParams& p, Feed& feed, int a, int n, const Turn& t, int from, float eps,
                                         int lane, __nv_bfloat16* out, int8_t* codes, float* scales, bool store) {
  uint4* dst = reinterpret_cast<uint4*>(out + (size_t)a * kHeadDim) + lane;
  if (kCodes) codes += a * kHeadDim, scales += a;
#pragma unroll 1
  for (; n > 0; n -= 4) {
    feed.fetch(p, lane);
    const uint32_t src = feed.slot();
    // rows i .. of the batch
    const auto do_some = [&](auto rows, int i, float e, float least_ok) {
      return do_rows<decltype(rows)::value, kTurn, kNorm, kCodes>(
          src + 512 * i, t, from, e, least_ok, lane, dst + i * (kHeadDim / 8), codes + (kCodes ? i * kHeadDim : 0),
          scales + (kCodes ? i : 0), store);
    };
    bool done = true;
    if (n >= 4) {
      done = do_some(Rows<4>{}, 0, eps, kTinyMeanSquare);
    } else {
      if (n >= 2) done = do_some(Rows<2>{}, 0, eps, kTinyMeanSquare);
      if (n & 1) done &= do_some(Rows<1>{}, n & 2, eps, kTinyMeanSquare);
    }
    if (__builtin_expect(!done, 0)) {
#pragma unroll 1
      for (int i = 0; i < min(n, 4); ++i) {
        float e = eps, least_ok = kTinyMeanSquare;
#pragma unroll 1
        while (!do_some(Rows<1>{}, i, e, least_ok)) {
          raise_row(src + 512 * i);
          e = e * kRaise * kRaise;
          least_ok = -1.f;
        }
      }
    }
    dst += 4 * (kHeadDim / 8);
    if (kCodes) codes += 4 * kHeadDim, scales += 4;
  }
}

// A warp takes items (token, part of its rows: queries, keys, values in turn)
// with a grid stride, rows four at a time.
template <bool kAppend, int kCap, int kTurn>
__global__ void __launch_bounds__(kQkvWarps * 32, kQkvPerSm) qkv_kernel(const __grid_constant__ QkvParams p,
                                                                        const __grid_constant__ QkvSeqs<kCap> tab) {
  __shared__ uint64_t turn[kMaxPairs];
  __shared__ int axis[kMaxPairs];
  __shared__ float2 cs_all[kQkvWarps][kMaxPairs];
  __shared__ __align__(16) uint4 ring[kQkvWarps][2 * 4 * kHeadDim / 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = kTurn == TURN_NONE ? 0 : p.rope.rot_dim / 2;
  if (kTurn != TURN_NONE) {
    for (int i = threadIdx.x; i < pairs; i += kQkvWarps * 32) {
      turn[i] = p.rope.turn[i];
      axis[i] = p.rope.axis[i];
    }
    __syncthreads();
  }
  float2* cs = cs_all[warp];
  const int hl = p.rope.rot_dim / 16;  // lanes of half the rotated dims
  const int from = lane < hl ? lane + hl : (lane < 2 * hl ? lane - hl : lane);
  const int n_rows = p.n_q + p.n_k + p.n_v;
  const long long n_items = (long long)p.n_tok * p.parts, stride = (long long)gridDim.x * kQkvWarps;
  struct Item {
    int row, tok, seq, r0, r1;
  };
  auto item_at = [&](long long item) {
    Item it;
    const int i = p.parts == 1 ? (int)item : (int)(item / p.parts);
    it.r0 = p.parts == 1 ? 0 : (int)(item - (long long)i * p.parts) * p.rows_per_part;
    it.r1 = min(n_rows, it.r0 + p.rows_per_part);
    it.row = it.tok = i;
    it.seq = 0;
    if (kAppend) {  // the launch's i-th token: its sequence, row and position
      if (p.same_len > 0) {
        it.seq = i / p.same_len;
      } else {
        int lo = 0, hi = p.n_seq - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (tab.s[mid].z <= i) lo = mid;
          else hi = mid - 1;
        }
        it.seq = lo;
      }
      const int4 s = tab.s[it.seq];
      it.row = s.x + (i - s.z);
      it.tok = s.y + (i - s.z);
    }
    return it;
  };
  long long item = (long long)blockIdx.x * kQkvWarps + warp;
  if (item >= n_items) return;
  Item now = item_at(item), then{};
  Feed feed{smem_u32(ring[warp]) + 16 * lane, 0, now.row, now.r0, now.r1, -1, 0, 0};
  feed.fetch(p, lane);
  for (; item < n_items; item += stride, now = then) {
    if (item + stride < n_items) {
      then = item_at(item + stride);
      feed.next_row = then.row, feed.next_r0 = then.r0, feed.next_r1 = then.r1;
    }
    const int row = now.row, tok = now.tok, seq = now.seq, r0 = now.r0, r1 = now.r1;
    int phys = -1;
    if (kAppend && r1 > p.n_q) {
      phys = __ldg(p.block_table + (size_t)(p.bt_row0 + seq) * p.bt_stride + tok / kPage);
      if (phys < 0 || phys >= p.n_pool) {  // never dereferenced
        if (lane == 0) record_bad_page(p.err);
        phys = -1;
      }
    }
    // cosine and sine of the token's angles, one per pair
    if (kTurn != TURN_NONE && r0 < p.n_q + p.n_k) {
      __syncwarp();  // every lane has read cs before
      for (int j = lane; j < pairs; j += 32) {
        const int pos = p.pos ? __ldg(p.pos + (size_t)axis[j] * p.pos_stride + row) : tok;
        const uint64_t frac = turn[j] * (uint64_t)(int64_t)pos;
        const float x = (float)(int32_t)((frac + 0x80000000ull) >> 32) * 4.656612873077393e-10f;  // 2^-31: half turns
        float sn, cn;
        sincospif(x, &sn, &cn);
        cs[j] = make_float2(cn, sn);
      }
      __syncwarp();
    }
    Turn t;
    if (r0 < p.n_q) {
      make_turn<kTurn>(p, p.qw, cs, lane, from, t);
      do_heads<kTurn, true, false>(p, feed, r0, min(r1, p.n_q) - r0, t, from, p.eps, lane,
                                   p.q_out + (size_t)row * p.n_q * kHeadDim, nullptr, nullptr, true);
    }
    const size_t slot = kAppend ? ((size_t)max(phys, 0) * kPage + tok % kPage) * p.HKV : 0;
    const int ka = max(r0 - p.n_q, 0), kb = min(r1 - p.n_q, p.n_k);
    if (ka < kb) {
      make_turn<kTurn>(p, p.kw, cs, lane, from, t);
      do_heads<kTurn, true, kAppend>(p, feed, ka, kb - ka, t, from, p.eps, lane, p.k_out + (size_t)row * p.n_k * kHeadDim,
                                     p.k_pool + slot * kHeadDim, p.k_scale + slot, phys >= 0);
    }
    if (kAppend) {
      const int va = max(r0 - p.n_q - p.n_k, 0), vb = r1 - p.n_q - p.n_k;
      if (va < vb)
        do_heads<TURN_NONE, false, true>(p, feed, va, vb - va, t, from, 0.f, lane, p.k_out, p.v_pool + slot * kHeadDim,
                                         p.v_scale + slot, phys >= 0);
    }
  }
}

template <bool kAppend, int kCap>
cudaError_t launch(const QkvParams& p, const QkvSeqs<kCap>& tab, int n_sm, cudaStream_t st) {
  const long long items = (long long)p.n_tok * p.parts;
  const long long want = (items + kQkvWarps - 1) / kQkvWarps, most = (long long)n_sm * kQkvPerSm;
  const int grid = (int)(want < most ? want : most);
  if (p.rope.rot_dim == 0) qkv_kernel<kAppend, kCap, TURN_NONE><<<grid, kQkvWarps * 32, 0, st>>>(p, tab);
  else if (p.rope.pairing == PA_ROPE_HALF) qkv_kernel<kAppend, kCap, TURN_HALVES><<<grid, kQkvWarps * 32, 0, st>>>(p, tab);
  else qkv_kernel<kAppend, kCap, TURN_ADJACENT><<<grid, kQkvWarps * 32, 0, st>>>(p, tab);
  return cudaGetLastError();
}

}  // namespace

// How many of a token's rows a warp takes at a time: the number whose last wave
// of items ends first.  An item costs its set-up (the token's page, its gains,
// sines and cosines) and its rows, four, two or one at a time; in units of a
// twentieth of the set-up, from batches of 300 to 32768 tokens (us, all sizes
// from one row to all tried).  300 tokens of 12 rows: 3.8 with four rows (5.4
// with all, 5.2 with one); 3000: 8.3 with all (10.5 with four); 9776 of 24: 41.6
// with all (57.3 with four, 58.0 with 16).
int qkv_rows_per_part(long long n_tok, int rows, int n_sm) {
  const long long warps = (long long)n_sm * kQkvPerSm * kQkvWarps;
  double best = 0.0;
  int per = 0;
  for (int r = 1;; r = r < 4 ? 2 * r : r + 4) {
    r = r < rows ? r : rows;
    const long long items = n_tok * ((rows + r - 1) / r), waves = (items + warps - 1) / warps;
    const double cost = (double)waves * (20 + 6 * (r / 4) + (r % 4 >= 2 ? 5 : 0) + (r % 2 ? 4 : 0)) + 6.0 * items / warps;
    if (per == 0 || cost < best) best = cost, per = r;
    if (r == rows) return per;
  }
}

cudaError_t launch_qk_norm_rope(const QkvParams& p, int n_sm, cudaStream_t st) {
  const QkvSeqs<1> none{};
  return launch<false, 1>(p, none, n_sm, st);
}

cudaError_t launch_qkv_append(const QkvParams& p, const QkvSeqs<kQkvSeqs>& seqs, int n_sm, cudaStream_t st) {
  if (p.n_seq <= kQkvFewSeqs) {
    QkvSeqs<kQkvFewSeqs> few;
    for (int i = 0; i < kQkvFewSeqs; ++i) few.s[i] = i < p.n_seq ? seqs.s[i] : make_int4(0, 0, 0, 0);
    return launch<true, kQkvFewSeqs>(p, few, n_sm, st);
  }
  return launch<true, kQkvSeqs>(p, seqs, n_sm, st);
}

}  // namespace pa
