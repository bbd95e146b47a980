// The paged 4-bit KV pool (sm_103a): the append of new rows, the rows read back,
// and the widening pass that feeds the prefill attention from it.
//
// A row x of 256 values (one token, one kv head, K or V) is held as e2m1 codes
// under e4m3 scales of 16 values each and one fp32 scale s:
//   s      the least power of two 2^e with max|x| <= 2688 2^e (2688 = 6 x 448, the
//          largest code times the largest block scale), e >= -100; 0 for a row of zeros
//   b_i    = e4m3(max over block i of |x| / (6 s))
//   code_d = e2m1(x_d / (b_i s)), 0 where b_i is 0; |.| > 6 gives 6
// each to nearest, ties to even.  code b_i has 6 significant bits, is a multiple of
// 2^-10 and at most 2688: exact in bf16 and in fp16, and x's value code b_i s in bf16.
//
// The decisions are exact for bf16 rows.  With s a power of two x / s is exact.  A
// bf16 maximum has 8 significant bits, and 6 times a border between two e4m3 values
// at most 7, so a quotient that is not a border is at least 2^-8 of its size away
// from one: the product with RN(1/6), off by 2^-23, rounds alike, and at a border the
// product is the border (checked for all significands).  Likewise x / (b s) is a
// border of e2m1 or 2^-8 of its size away from it; x r with r near 1 / (b s) would
// miss a border that it should meet, so it is rounded to a multiple of 2^-13 first,
// by adding and taking away 1536 = 1.5 x 2^10: what lies within 2^-14 of a border
// becomes the border, and nothing else crosses one.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pa_internal.h"
#include "pa_kv4.cuh"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kRowsWarps = 8;
constexpr long long kFewWarps = 8192;  // below as many (token, kv head) rows a warp takes one
constexpr unsigned kAll = 0xffffffffu;

// Sequence and token of the launch's i-th token: its row, position and block-table row.
struct Tok {
  int row, tok, seq;
};
template <int kCap>
__device__ __forceinline__ Tok token_at(const Kv4RowsParams& p, const QkvSeqs<kCap>& tab, int i) {
  int s;
  if (p.same_len > 0) {
    s = i / p.same_len;
  } else {
    int lo = 0, hi = p.n_seq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.s[mid].z <= i) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
  }
  const int4 e = tab.s[s];
  return Tok{e.x + (i - e.z), e.y + (i - e.z), s};
}

__device__ __forceinline__ uint32_t absmax_bits8(const uint4 raw) {
  const uint32_t m = __vmaxu2(__vmaxu2(raw.x & 0x7fff7fffu, raw.y & 0x7fff7fffu),
                              __vmaxu2(raw.z & 0x7fff7fffu, raw.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// Of a row's largest magnitude (bf16 bits): the biased exponent of s, at least 27 (2^-100).
__device__ __forceinline__ int step_exponent(uint32_t am) {
  // 2688 = 1.3125 x 2^11, and 1.3125 is significand 40 of 128
  return max(27, (int)(am >> 7) - 11 + ((am & 127u) > 40u ? 1 : 0));
}

// A lane's eight values as codes, r = 1 / (b s) or 0.
__device__ __forceinline__ uint32_t codes8(const uint4 raw, float r) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float y[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 v = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    v = add2(fma2(v, make_float2(r, r), make_float2(1536.f, 1536.f)), make_float2(-1536.f, -1536.f));
    y[2 * j] = v.x;
    y[2 * j + 1] = v.y;
  }
  return to_e2m1x8(y);
}

// Bound by memory (512 bytes in and 148 out a row) and nearly by its arithmetic: 9777
// tokens of 8 heads, 103 MB, 18.4 us (5.6 TB/s; ALU pipe 64 % busy); with one head a warp 23.8,
// two 20.9 (the token's sequence and page are looked up again for each); the other way, the
// gather, 18.0 against 20.4 and 18.3.  Few rows take one head a warp: 64 tokens 1.7 us.
// A warp takes kHeads kv heads of a token, K and V rows of each, eight values a lane of
// every row, all rows' loads in flight with the block-table read.
template <int kCap, int kHeads>
__global__ void __launch_bounds__(kRowsWarps * 32) kv4_append_kernel(const __grid_constant__ Kv4RowsParams p,
                                                                     const __grid_constant__ QkvSeqs<kCap> tab) {
  const int i = blockIdx.x * kRowsWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31, g0 = blockIdx.y * kHeads;
  dependents_may_start();
  if (i >= p.n_tok) return;
  const Tok t = token_at(p, tab, i);
  wait_for_previous();
  const __nv_bfloat16* k = p.k.p + (size_t)t.row * p.k.ts + (size_t)g0 * p.k.hs + 8 * lane;
  const __nv_bfloat16* v = p.v.p + (size_t)t.row * p.v.ts + (size_t)g0 * p.v.hs + 8 * lane;
  uint4 rk[kHeads], rv[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    const bool have = kHeads == 1 || g0 + h < p.HKV;
    rk[h] = have ? __ldcg(reinterpret_cast<const uint4*>(k + (size_t)h * p.k.hs)) : make_uint4(0u, 0u, 0u, 0u);
    rv[h] = have ? __ldcg(reinterpret_cast<const uint4*>(v + (size_t)h * p.v.hs)) : make_uint4(0u, 0u, 0u, 0u);
  }
  const int phys = __ldcg(p.block_table + (size_t)(p.bt_row0 + t.seq) * p.bt_stride + t.tok / kPage);
  if (phys < 0 || phys >= p.n_pool) {  // never dereferenced
    if (lane == 0) record_bad_page(p.err);
    return;
  }
  const int r = t.tok % kPage, at = kv4_piece(r, lane >> 2) + 4 * (lane & 3);
  uint8_t* tile = p.pool + ((size_t)phys * p.HKV + g0) * kT4Bytes;
#pragma unroll
  for (int h = 0; h < kHeads; ++h, tile += kT4Bytes) {
    if (kHeads > 1 && g0 + h >= p.HKV) break;
    // the largest magnitudes of K and V as the halves of one word: over the block (two lanes), then the row
    uint32_t m = absmax_bits8(rk[h]) | (absmax_bits8(rv[h]) << 16);
    m = __vmaxu2(m, __shfl_xor_sync(kAll, m, 1));
    const uint32_t mb = m;
#pragma unroll
    for (int o = 2; o < 32; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(kAll, m, o));
    const int ek = step_exponent(m & 0xffffu), ev = step_exponent(m >> 16);
    const float ik = __uint_as_float((uint32_t)(254 - ek) << 23), iv = __uint_as_float((uint32_t)(254 - ev) << 23);
    constexpr float kSixth = 1.f / 6.f;
    const uint32_t b = to_e4m3x2(__uint_as_float(mb << 16) * ik * kSixth, __uint_as_float(mb & 0xffff0000u) * iv * kSixth);
    const uint32_t bh = e4m3x2_to_f16(b);
    const float2 bf = __half22float2(*reinterpret_cast<const __half2*>(&bh));
    float qk = 0.f, qv = 0.f;
    if (bf.x > 0.f) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(qk) : "f"(bf.x));
    if (bf.y > 0.f) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(qv) : "f"(bf.y));
    *reinterpret_cast<uint32_t*>(tile + at) = codes8(rk[h], qk * ik);
    *reinterpret_cast<uint32_t*>(tile + kT4V + at) = codes8(rv[h], qv * iv);
    if ((lane & 1) == 0) {
      tile[kT4Block + r * 16 + (lane >> 1)] = (uint8_t)(b & 0xffu);
      tile[kT4Block + 256 + r * 16 + (lane >> 1)] = (uint8_t)(b >> 8);
    }
    if (lane == 0) {
      *reinterpret_cast<float*>(tile + kT4Row + 4 * r) = (m & 0xffffu) ? __uint_as_float((uint32_t)ek << 23) : 0.f;
      *reinterpret_cast<float*>(tile + kT4Row + 64 + 4 * r) = (m >> 16) ? __uint_as_float((uint32_t)ev << 23) : 0.f;
    }
  }
}

// A lane's eight values of a row, code x block scale (exact in fp16) x row scale, to bf16.
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t block, float s) {
  uint32_t h[4], o[4];
  e2m1x8_to_f16(codes, h);
  const uint32_t b = __byte_perm(e4m3x2_to_f16(block), 0u, 0x1010);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = mul_f16x2(h[j], b);
    const __nv_bfloat162 v = __float22bfloat162_rn(mul2(__half22float2(*reinterpret_cast<const __half2*>(&x)), make_float2(s, s)));
    o[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int kCap, int kHeads>
__global__ void __launch_bounds__(kRowsWarps * 32) kv4_gather_kernel(const __grid_constant__ Kv4RowsParams p,
                                                                     const __grid_constant__ QkvSeqs<kCap> tab) {
  const int i = blockIdx.x * kRowsWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31, g0 = blockIdx.y * kHeads;
  dependents_may_start();
  if (i >= p.n_tok) return;
  const Tok t = token_at(p, tab, i);
  wait_for_previous();
  const int phys = __ldcg(p.block_table + (size_t)(p.bt_row0 + t.seq) * p.bt_stride + t.tok / kPage);
  if (phys < 0 || phys >= p.n_pool) {  // never dereferenced
    if (lane == 0) record_bad_page(p.err);
    return;
  }
  const int r = t.tok % kPage, at = kv4_piece(r, lane >> 2) + 4 * (lane & 3);
  const uint8_t* tile = p.pool + ((size_t)phys * p.HKV + g0) * kT4Bytes;
  uint32_t ck[kHeads], cv[kHeads], bk[kHeads], bv[kHeads];
  float sk[kHeads], sv[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (kHeads > 1 && g0 + h >= p.HKV) break;
    const uint8_t* th = tile + h * kT4Bytes;
    ck[h] = __ldcg(reinterpret_cast<const uint32_t*>(th + at));
    cv[h] = __ldcg(reinterpret_cast<const uint32_t*>(th + kT4V + at));
    bk[h] = __ldcg(th + kT4Block + r * 16 + (lane >> 1));
    bv[h] = __ldcg(th + kT4Block + 256 + r * 16 + (lane >> 1));
    sk[h] = __ldcg(reinterpret_cast<const float*>(th + kT4Row + 4 * r));
    sv[h] = __ldcg(reinterpret_cast<const float*>(th + kT4Row + 64 + 4 * r));
  }
  const size_t out = ((size_t)t.row * p.HKV + g0) * (kHeadDim / 8) + lane;
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (kHeads > 1 && g0 + h >= p.HKV) break;
    if (p.k_out) reinterpret_cast<uint4*>(p.k_out)[out + h * (kHeadDim / 8)] = values8(ck[h], bk[h], sk[h]);
    if (p.v_out) reinterpret_cast<uint4*>(p.v_out)[out + h * (kHeadDim / 8)] = values8(cv[h], bv[h], sv[h]);
  }
}

template <int N>
struct Heads {
  static constexpr int value = N;
};
// launch(grid, table, heads of a warp): HEADS
template <typename F>
cudaError_t with_table(const Kv4RowsParams& p, const QkvSeqs<kQkvSeqs>& seqs, F launch) {
  const unsigned x = (unsigned)((p.n_tok + kRowsWarps - 1) / kRowsWarps);
  const auto with_heads = [&](const auto& tab) {
    const long long warps = (long long)p.n_tok * p.HKV;
    if (p.HKV == 1 || warps < kFewWarps) return launch(dim3(x, p.HKV), tab, Heads<1>{});
    if (p.HKV <= 2) return launch(dim3(x, 1), tab, Heads<2>{});
    return launch(dim3(x, (p.HKV + 3) / 4), tab, Heads<4>{});
  };
  if (p.n_seq <= kQkvFewSeqs) {
    QkvSeqs<kQkvFewSeqs> few;
    for (int i = 0; i < kQkvFewSeqs; ++i) few.s[i] = i < p.n_seq ? seqs.s[i] : make_int4(0, 0, 0, 0);
    return with_heads(few);
  }
  return with_heads(seqs);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowsParams& p, const QkvSeqs<kQkvSeqs>& seqs, cudaStream_t st) {
  return with_table(p, seqs, [&](dim3 grid, const auto& tab, auto heads) {
    return launch_early(kv4_append_kernel<sizeof(tab.s) / sizeof(int4), decltype(heads)::value>, grid, kRowsWarps * 32, 0, st, p, tab);
  });
}
cudaError_t launch_kv4_gather(const Kv4RowsParams& p, const QkvSeqs<kQkvSeqs>& seqs, cudaStream_t st) {
  return with_table(p, seqs, [&](dim3 grid, const auto& tab, auto heads) {
    return launch_early(kv4_gather_kernel<sizeof(tab.s) / sizeof(int4), decltype(heads)::value>, grid, kRowsWarps * 32, 0, st, p, tab);
  });
}

// ======================================================================
// Widening: visible pages -> contiguous K (bf16, code x block scale, exact) and
// V^T (fp16, exact), with the row scales as the attention's per-token scales.
// One CTA per stored 16-token block, as widen_kernel has it; bound by latencies and by
// its stores, 16 KB a block and head into L2: 1025 blocks of two heads 12 us.
// ======================================================================
namespace {
constexpr int kWidenThreads = 256;

// Two lanes' 32 bytes each, the even lane's to `even` and the odd one's to `odd`, with
// both lanes on the same 32 bytes in each of the two stores (a lane storing its own
// halves in turn would write every sector twice by half).
__device__ __forceinline__ void store_pair(const uint32_t (&o)[8], uint4* even, uint4* odd, bool is_odd) {
  uint32_t other[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) other[j] = __shfl_xor_sync(kAll, is_odd ? o[j] : o[4 + j], 1);
  even[is_odd] = is_odd ? make_uint4(other[0], other[1], other[2], other[3]) : make_uint4(o[0], o[1], o[2], o[3]);
  odd[is_odd] = is_odd ? make_uint4(o[4], o[5], o[6], o[7]) : make_uint4(other[0], other[1], other[2], other[3]);
}

template <int HKV>
__global__ void __launch_bounds__(kWidenThreads) kv4_widen_kernel(const __grid_constant__ WidenParams p, const uint8_t* pool) {
  constexpr int kVWords = (2048 + 256) / 16;  // V's codes and block scales of a tile
  constexpr int kVLoads = (HKV * kVWords + kWidenThreads - 1) / kWidenThreads;
  __shared__ uint4 v_sh[HKV * kVWords];
  __shared__ unsigned int vmax_sh[2 * HKV];  // the largest V scale's bits, 0x7f800000 - the least's
  const int blk = blockIdx.x, tid = threadIdx.x;
  dependents_may_start();
  if (tid < 2 * HKV) vmax_sh[tid] = 0u;
  wait_for_previous();
  // the block's sequence: the last one that starts at or before it
  int s = -1;
  for (int s0 = 0; s0 < p.n_seq; s0 += kWidenThreads) {
    const int n = __syncthreads_count(s0 + tid < p.n_seq && p.seqs[min(s0 + tid, p.n_seq - 1)].tok_off <= blk * kPage);
    s += n;
    if (n < kWidenThreads) break;
  }
  const SeqGeom sg = p.seqs[s];
  const int kb = stored_to_logical_block(sg, blk - sg.tok_off / kPage);
  const int row0 = blk * kPage;
  const int phys = p.block_table[(size_t)sg.bt_row * p.bt_stride + kb];
  const bool bad = phys < 0 || phys >= p.n_pool;
  if (bad && tid == 0) record_bad_page(p.err);
  const int n_valid = bad ? 0 : imax(0, imin(kPage, sg.n_ctx - kb * kPage));
  const uint8_t* page = pool + (size_t)(bad ? 0 : phys) * HKV * kT4Bytes;
  // every load of the block before its first store: V's codes and block scales, K's 16 dims (a block) a thread
  // and head, the row scales of thread tid < 16 HKV's token and head
  uint4 vr[kVLoads];
#pragma unroll
  for (int i = 0; i < kVLoads; ++i) {
    const int w = tid + kWidenThreads * i, g = w / kVWords, k = w % kVWords;
    vr[i] = make_uint4(0u, 0u, 0u, 0u);
    if (w < HKV * kVWords && !bad)
      vr[i] = __ldcg(reinterpret_cast<const uint4*>(page + g * kT4Bytes + (k < 128 ? kT4V : kT4Block + 256 - 2048)) + k);
  }
  const int kr_ = tid >> 4, kb_ = tid & 15;  // K: token, block of dims
  uint2 kw[HKV];
  uint32_t ksc[HKV];
#pragma unroll
  for (int g = 0; g < HKV; ++g) {
    kw[g] = make_uint2(0u, 0u);
    ksc[g] = 0u;
    if (kr_ < n_valid) {
      const uint8_t* tile = page + g * kT4Bytes;
      kw[g] = __ldcg(reinterpret_cast<const uint2*>(tile + kv4_piece(kr_, kb_ >> 1) + 8 * (kb_ & 1)));
      ksc[g] = __ldcg(tile + kT4Block + kr_ * 16 + kb_);
    }
  }
  float ks_row = 0.f, vs_row = 0.f;
  if (tid < kPage * HKV && (tid & 15) < n_valid) {
    const float* row = reinterpret_cast<const float*>(page + (tid >> 4) * kT4Bytes + kT4Row) + (tid & 15);
    ks_row = __ldcg(row);
    vs_row = __ldcg(row + 16);
  }
#pragma unroll
  for (int i = 0; i < kVLoads; ++i)
    if (tid + kWidenThreads * i < HKV * kVWords) v_sh[tid + kWidenThreads * i] = vr[i];
#pragma unroll
  for (int g = 0; g < HKV; ++g) {
    const uint32_t sc = __byte_perm(e4m3x2_to_f16(ksc[g]), 0u, 0x1010);
    uint32_t h[8], o[8];
    e2m1x8_to_f16(kw[g].x, reinterpret_cast<uint32_t(&)[4]>(h[0]));
    e2m1x8_to_f16(kw[g].y, reinterpret_cast<uint32_t(&)[4]>(h[4]));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t x = mul_f16x2(h[j], sc);
      const __nv_bfloat162 v = __float22bfloat162_rn(__half22float2(*reinterpret_cast<const __half2*>(&x)));
      o[j] = *reinterpret_cast<const uint32_t*>(&v);
    }
    uint4* dst = reinterpret_cast<uint4*>(p.kw + ((size_t)g * p.n_tok_cap + row0 + kr_) * kHeadDim + (kb_ & 14) * 16);
    store_pair(o, dst, dst + 2, tid & 1);
  }
  __syncthreads();
  // V: two dims (a byte of each token's codes) a thread and turn, their 16 tokens' columns
  for (int i = tid; i < HKV * (kHeadDim / 2); i += kWidenThreads) {
    const int d2 = i & 127, g = i >> 7;
    const uint8_t* codes = reinterpret_cast<const uint8_t*>(v_sh + g * kVWords);
    uint32_t x[16];
#pragma unroll
    for (int r = 0; r < kPage; ++r) {
      x[r] = 0u;
      if (r < n_valid) {
        uint32_t h;
        const uint32_t c = codes[kv4_piece(r, d2 >> 4) + (d2 & 15)];
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h) : "r"(c));
        x[r] = mul_f16x2(h, __byte_perm(e4m3x2_to_f16(codes[2048 + r * 16 + (d2 >> 3)]), 0u, 0x1010));
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = __byte_perm(x[2 * j], x[2 * j + 1], e ? 0x7632 : 0x5410);
      __half* row = p.vt + ((size_t)g * kHeadDim + 2 * (d2 & ~1) + e) * p.n_tok_cap + row0;
      store_pair(o, reinterpret_cast<uint4*>(row), reinterpret_cast<uint4*>(row + 2 * (size_t)p.n_tok_cap), tid & 1);
    }
  }
  // scales (0 past the end of the context), the largest V scale and the least
  if (tid < kPage * HKV) {
    const int r = tid & 15, g = tid >> 4;
    p.ks[(size_t)g * p.n_tok_cap + row0 + r] = ks_row * p.k_mult;
    p.vs[(size_t)g * p.n_tok_cap + row0 + r] = vs_row;
    if (r < n_valid) {
      atomicMax(&vmax_sh[g], __float_as_uint(vs_row));
      atomicMax(&vmax_sh[HKV + g], 0x7f800000u - __float_as_uint(vs_row));
    }
  }
  __syncthreads();
  if (tid < 2 * HKV) {
    const unsigned int m = vmax_sh[tid];
    unsigned int* gm = p.vsmax + (tid < HKV ? s * HKV + tid : (p.n_seq + s) * HKV + tid - HKV);
    if (m > *reinterpret_cast<volatile unsigned int*>(gm)) atomicMax(gm, m);
  }
}
// The largest and least V scales before the widening raises them (a kernel and not a memset: the widening
// is then set up early too; 2 us of a call of few tokens).  The widening may start behind the wait
// only: with the last call's attention on most SMs its CTAs would crowd on the others.
__global__ void __launch_bounds__(256) zero_kernel(unsigned int* x, int n) {
  wait_for_previous();
  dependents_may_start();
  for (int i = threadIdx.x; i < n; i += 256) x[i] = 0u;
}

template <int HKV>
cudaError_t launch_widen(const WidenParams& p, const uint8_t* pool, cudaStream_t st) {
  const cudaError_t e = launch_early(zero_kernel, dim3(1), 256, 0, st, p.vsmax, 2 * p.n_seq * HKV);
  if (e != cudaSuccess) return e;
  return launch_early(kv4_widen_kernel<HKV>, dim3((unsigned)p.n_stored_blocks), kWidenThreads, 0, st, p, pool);
}
}  // namespace

cudaError_t launch_widen_kv4(const WidenParams& p, const uint8_t* pool, cudaStream_t st) {
  switch (p.HKV) {
    case 1: return launch_widen<1>(p, pool, st);
    case 2: return launch_widen<2>(p, pool, st);
    case 3: return launch_widen<3>(p, pool, st);
    case 4: return launch_widen<4>(p, pool, st);
    case 5: return launch_widen<5>(p, pool, st);
    case 6: return launch_widen<6>(p, pool, st);
    case 7: return launch_widen<7>(p, pool, st);
    case 8: return launch_widen<8>(p, pool, st);
    default: return cudaErrorInvalidValue;  // the handle accepts 1..8 kv heads
  }
}

}  // namespace pa
