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
// 64-bit binary fraction F instead; position * F mod 2^64 is the exact
// fraction of a turn, in one integer product, and the sine and cosine are
// taken of that fraction (|x| <= 1 half turn, error 2^-25 of one).
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

constexpr int kQkvWarps = 8;
constexpr int kMaxPairs = kHeadDim / 2;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void unpack8(const uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(u[j] << 16);
    x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
    u[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// Where a lane's rotation partners are.  The lane holds dims [8 lane, 8 lane +
// 8).  Halves: dim i < R/2 pairs with i + R/2, a whole lane R/16 lanes away (R
// is a multiple of 16).  Neighbours: dims 2i and 2i + 1, in the same word.
struct Partner {
  int lane;
  bool halves;
  __device__ __forceinline__ uint32_t word(uint32_t w) const {
    return halves ? __shfl_sync(kAll, w, lane) : __byte_perm(w, w, 0x1032);
  }
  __device__ __forceinline__ uint4 words(const uint4 w) const {
    return make_uint4(word(w.x), word(w.y), word(w.z), word(w.w));
  }
};

// A and B of the lane's eight dims for one set of gains.
struct Turn {
  float a[8], b[8];
};
__device__ __forceinline__ void make_turn(const QkvParams& p, const __nv_bfloat16* w, const float2* cs, int lane,
                                          const Partner& pt, Turn& t) {
  float g[8], gp[8];
  if (w) {
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(w) + lane);
    unpack8(raw, g);
    unpack8(pt.words(raw), gp);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] += p.w_off, gp[e] += p.w_off;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = gp[e] = 1.f;
  }
  const int d0 = 8 * lane, R = p.rope.rot_dim;
#pragma unroll
  for (int e = 0; e < 8; ++e) t.a[e] = g[e], t.b[e] = 0.f;
  if (d0 < R) {
    const int half = R / 2;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool first = pt.halves ? d0 < half : (e & 1) == 0;
      const float2 c = cs[pt.halves ? (d0 < half ? d0 : d0 - half) + e : (d0 + e) >> 1];
      t.a[e] = g[e] * c.x;
      t.b[e] = first ? -gp[e] * c.y : gp[e] * c.y;
    }
  }
}

// The lane's eight values of a row, normed and turned.
__device__ __forceinline__ void norm_turn(const uint4 raw, const Turn& t, const Partner& pt, bool rotate, float eps,
                                          float (&y)[8]) {
  float x[8];
  unpack8(raw, x);
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
  const float ms = warp_sum(ss) * (1.f / kHeadDim) + eps;
  const float r = ms > 0.f ? rsqrtf(ms) : 0.f;  // an all-zero row with eps 0 stays zero
  if (rotate) {
    float xp[8];
    unpack8(pt.words(raw), xp);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = r * fmaf(xp[e], t.b[e], x[e] * t.a[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = r * (x[e] * t.a[e]);
  }
}

// One row into the pool: scale = absmax / 127, codes rint(x / scale) half to
// even, decided on the IEEE quotient as kv_append_kernel decides them.  x *
// rcp, rcp the hardware reciprocal, is within 3.1e-5 of that quotient
// (|quotient| <= 127.5), so only quotients within 1e-4 of a half-integer take
// the division; adding 1.5 * 2^23 rounds the others and leaves the code in the
// sum's low byte.  Rows with a subnormal scale, which the approximate
// reciprocal flushes, take the division too.
__device__ __forceinline__ void store_codes(const float (&x)[8], int lane, int8_t* codes, float* scale_out) {
  float am = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(x[e]));
  am = warp_max(am);
  const float scale = __fdiv_rn(am, 127.f);
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23
  float rcp = 0.f;
  if (scale > 0.f) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rcp) : "f"(scale));
  uint32_t f[8];
  float dmax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q = x[e] * rcp, s = q + kRound;
    dmax = fmaxf(dmax, fabsf(q - (s - kRound)));
    f[e] = __float_as_uint(s);
  }
  if (dmax > 0.4999f || (scale > 0.f && scale < 1.17549435e-38f)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __float_as_uint(rintf(__fdiv_rn(x[e], scale)) + kRound);
  }
  const uint32_t lo = __byte_perm(__byte_perm(f[0], f[1], 0x0040), __byte_perm(f[2], f[3], 0x0040), 0x5410);
  const uint32_t hi = __byte_perm(__byte_perm(f[4], f[5], 0x0040), __byte_perm(f[6], f[7], 0x0040), 0x5410);
  reinterpret_cast<uint2*>(codes)[lane] = make_uint2(lo, hi);
  if (lane == 0) *scale_out = scale;
}

enum : int { KIND_Q, KIND_K, KIND_V };

// A warp takes items (token, part of its rows) with a grid stride.  Rows go
// four at a time, all their loads before the first is used.
constexpr int kBatch = 4;

template <bool kAppend, int kCap>
__global__ void __launch_bounds__(kQkvWarps * 32) qkv_kernel(const __grid_constant__ QkvParams p,
                                                             const __grid_constant__ QkvSeqs<kCap> tab) {
  __shared__ uint64_t turn[kMaxPairs];
  __shared__ int axis[kMaxPairs];
  __shared__ float2 cs_all[kQkvWarps][kMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = p.rope.rot_dim / 2;
  for (int i = threadIdx.x; i < pairs; i += kQkvWarps * 32) {
    turn[i] = p.rope.turn[i];
    axis[i] = p.rope.axis[i];
  }
  __syncthreads();
  float2* cs = cs_all[warp];
  Partner pt;
  pt.halves = p.rope.pairing == PA_ROPE_HALF;
  const int hl = p.rope.rot_dim / 16;  // lanes of half the rotated dims
  pt.lane = lane < hl ? lane + hl : (lane < 2 * hl ? lane - hl : lane);
  const int n_rows = p.n_q + p.n_k + p.n_v;
  const long long n_items = (long long)p.n_tok * p.parts;
  for (long long item = (long long)blockIdx.x * kQkvWarps + warp; item < n_items;
       item += (long long)gridDim.x * kQkvWarps) {
    const int i = (int)(item / p.parts);
    const int r0 = (int)(item % p.parts) * p.rows_per_part, r1 = min(n_rows, r0 + p.rows_per_part);
    int row = i, tok = i, seq = 0;
    if (kAppend) {  // the launch's i-th token: its sequence, row and position
      if (p.same_len > 0) {
        seq = i / p.same_len;
      } else {
        int lo = 0, hi = p.n_seq - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (tab.s[mid].z <= i) lo = mid;
          else hi = mid - 1;
        }
        seq = lo;
      }
      const int4 s = tab.s[seq];
      row = s.x + (i - s.z);
      tok = s.y + (i - s.z);
    }
    // cosine and sine of the token's angles, one per pair
    const bool turned = pairs > 0 && r0 < p.n_q + p.n_k;
    if (turned) {
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
    int phys = -1;
    if (kAppend && r1 > p.n_q) {
      phys = __ldg(p.block_table + (size_t)(p.bt_row0 + seq) * p.bt_stride + tok / kPage);
      if (phys < 0 || phys >= p.n_pool) {  // never dereferenced
        if (lane == 0) atomicCAS(p.err, 0, DEV_ERR_BAD_PAGE);
        phys = -1;
      }
    }
    Turn t;
    for (int kind = KIND_Q; kind <= (kAppend ? KIND_V : KIND_K); ++kind) {
      const int base = kind == KIND_Q ? 0 : (kind == KIND_K ? p.n_q : p.n_q + p.n_k);
      const int cnt = kind == KIND_Q ? p.n_q : (kind == KIND_K ? p.n_k : p.n_v);
      const int a = max(r0 - base, 0), b = min(r1 - base, cnt);  // heads of this kind
      if (a >= b) continue;
      const RowsIn in = kind == KIND_Q ? p.q : (kind == KIND_K ? p.k : p.v);
      const uint4* src = reinterpret_cast<const uint4*>(in.p + (size_t)row * in.ts) + lane;
      const size_t hstep = (size_t)in.hs / 8;
      bool made = kind == KIND_V;
      for (int h0 = a; h0 < b; h0 += kBatch) {
        uint4 raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (h0 + u < b) raw[u] = src[(size_t)(h0 + u) * hstep];
        if (!made) {
          make_turn(p, kind == KIND_Q ? p.qw : p.kw, cs, lane, pt, t);
          made = true;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (h0 + u >= b) break;
          const int h = h0 + u;
          float y[8];
          if (kind == KIND_V) unpack8(raw[u], y);
          else norm_turn(raw[u], t, pt, pairs > 0, p.eps, y);
          if (kind == KIND_Q) {
            reinterpret_cast<uint4*>(p.q_out + ((size_t)row * p.n_q + h) * kHeadDim)[lane] = pack8(y);
          } else if (!kAppend) {
            reinterpret_cast<uint4*>(p.k_out + ((size_t)row * p.n_k + h) * kHeadDim)[lane] = pack8(y);
          } else if (phys >= 0) {
            const size_t slot = ((size_t)phys * kPage + tok % kPage) * p.HKV + h;
            if (kind == KIND_K) store_codes(y, lane, p.k_pool + slot * kHeadDim, p.k_scale + slot);
            else store_codes(y, lane, p.v_pool + slot * kHeadDim, p.v_scale + slot);
          }
        }
      }
    }
    if (turned) __syncwarp();  // every lane has read cs before the next item's
  }
}

template <bool kAppend, int kCap>
cudaError_t launch(const QkvParams& p, const QkvSeqs<kCap>& tab, int n_sm, cudaStream_t st) {
  const long long items = (long long)p.n_tok * p.parts;
  const long long want = (items + kQkvWarps - 1) / kQkvWarps;
  const int grid = (int)(want < (long long)n_sm * 8 ? want : (long long)n_sm * 8);
  qkv_kernel<kAppend, kCap><<<grid, kQkvWarps * 32, 0, st>>>(p, tab);
  return cudaGetLastError();
}

}  // namespace

int qkv_rows_per_part(long long n_tok, int rows, int n_sm) {
  const long long warps = (long long)n_sm * 16;
  const long long per = (n_tok * rows + warps - 1) / warps;
  const int want = (int)(per < rows ? (per < 1 ? 1 : per) : rows);
  const int parts = (rows + want - 1) / want;
  return (rows + parts - 1) / parts;
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
