// Decode of a batch that shares a long prefix (sm_103a): one new query token
// per sequence, the first keys of every sequence the same pages of the pool.
//
// Softmax over the visible keys splits over any partition of them: with
// (m, l, O) the reference, sum and unnormalised output of a part,
//   m = max m_i,  l = sum 2^(m_i - m) l_i,  O = sum 2^(m_i - m) O_i.
// Up to three launches:
//   prefix_*_kernel  the prefix's keys against the queries of ALL sequences: per
//                    kv head a matrix of n_seq x G rows, so its K and V codes
//                    are read once and the products run on the tensor cores
//                    (tcgen05) instead of once per sequence
//   own_kernel       each sequence's own keys (with few sequences or a short
//                    prefix, all its keys), split into chunks
//   merge_kernel     the partials of both, and the division
//
// The prefix pass.  The int8 codes are widened to fp16 (exact) on their way into
// shared memory, K and V alike as [key][64 dims] rows of 128 bytes: a K-major B
// operand for S = Q K^T and an MN-major one for O = P V, so V needs no transpose.
// Scores, softmax and P' are those of the decode kernel: the bf16 query enters as
// fp16 through a power of two per row, P' = p * v_scale * 2^-e in fp16 (11 bits
// against the 8 of the output), fp32 sums.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "pa_shared.h"

namespace pa {
namespace {

constexpr unsigned kAllLanes = 0xffffffffu;
// The softmax reference moves when a row's maximum passes it by more than 2^15
// (moving it rescales O, ~1500 cycles); P' <= 2^15 then, inside fp16's range.
constexpr float kMaxLift = 15.f;
constexpr int DEV_ERR_LAYOUT = 0x400;  // shared memory's base is not aligned as the operands need (reported as PA_ECUDA)
constexpr uint64_t kShDrainNs = 200000000ull;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int N>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Four codes (bytes) -> two words of fp16 pairs: (b ^ 0x80) in the low byte of
// 0x64__ is 1152 + b, and the subtraction is exact.
__device__ __forceinline__ uint32_t minus_1152(uint32_t u) {
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480u)));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t lo_pair(uint32_t flipped) { return minus_1152(__byte_perm(flipped, 0x64646464u, 0x5140)); }
__device__ __forceinline__ uint32_t hi_pair(uint32_t flipped) { return minus_1152(__byte_perm(flipped, 0x64646464u, 0x7362)); }
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Volatile, so that it stays behind the wait that made the data visible.
__device__ __forceinline__ uint4 lds_u32x4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// 16 TMEM lanes x 128 columns in the 16x256b shape (see pa_ptx.cuh).
__device__ __forceinline__ void tmem_st_16x256b_x16(uint32_t taddr, const uint32_t (&r)[64]) {
#define PA_SH_W8(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,%64};" ::"r"(taddr),
      PA_SH_W8(0), PA_SH_W8(8), PA_SH_W8(16), PA_SH_W8(24), PA_SH_W8(32), PA_SH_W8(40), PA_SH_W8(48), PA_SH_W8(56)
      : "memory");
#undef PA_SH_W8
}
// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// e with 2^(e-1) <= x < 2^e, in [-100, 100]; -100 for x <= 0.
__device__ __forceinline__ int exp_above(float x) {
  return x > 0.f ? max(-100, min(100, (int)((__float_as_uint(x) >> 23) & 0xff) - 126)) : -100;
}
// The exponent k of the power of two that puts a row's absolute maximum in [64, 128).
__device__ __forceinline__ int row_shift(float am) {
  return am > 0.f ? min(127, 133 - (int)((__float_as_uint(am) >> 23) & 0xff)) : 0;
}
__device__ __forceinline__ void unpack8(const uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(u[j] << 16);
    x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
  }
}

// ====================================================================
// The prefix
// ====================================================================
// kN = 2, more than 128 query rows a kv head: a pair of SMs (cluster of two CTAs)
// computes groups of 256 rows, 128 in each CTA's TMEM, against tiles of 128 keys;
// one thread of the even CTA issues every product of both (cta_group::2).  The B
// operands are split: each CTA holds K of 64 of a tile's keys and V of 128 of the
// 256 dims, so it reads and widens half of every tile's codes, which (with one CTA
// per tile: 64 KB of codes read, 128 KB of operands written and 192 KB of operands
// read per tile and SM) would otherwise bound the kernel.
// kN = 1, up to 128 rows: a pair's second CTA would have none.  Each CTA takes
// whole tiles by itself: K in two parts of 128 dims and V in two of 64 keys, one
// stage for each, so that a part is widened while the other one's products run.
// (9 sequences of 8 rows on 131072 keys: 33 us, with 64-key tiles in double stages
// 35, on pairs 40; 12 on 16384: 21, 20, 22.)
//
// What bounds it.  64 sequences, 16 q and 2 kv heads, 32768 keys: 51 us, 18 tiles
// a pair of ~3500 cycles each, between 11000 of set-up and 5500 of storing partials.
// The tensor pipe runs 2048 of a tile's cycles.  The rest is the chain from scores
// to products: softmax (~2000), an arrival from the other CTA (300 to 1100), the
// issue of the products (70 to 90 cycles each), and in most tiles some warp that
// moves a reference and rescales O (~1500; without outlier keys, 50.5 us instead
// of 53.4 at the time).  A CTA alone: ~5000 cycles a tile, all of whose codes it
// widens itself, beside the same softmax.
// Tried and not better: two sets of softmax warps in turn, 16 of them on half of
// the keys each, warps of their own for the rescale (all: more warps, each
// slower), a thread each for Q K^T and P V (what runs in order on one thread then
// waits for the other's commit), and prefetches of later tiles' codes into L2.
constexpr int kSoftWarps = 8;                       // warps 0-7: softmax; TMEM quadrant w % 4, 16 rows w / 4 of it
constexpr int kConvWarps = 8;                       // warps 8-15: codes -> fp16 operands (K: four, V: four), the queries
constexpr int kIssueWarp = kSoftWarps + kConvWarps; // warp 16: TMEM; even CTA: the products, odd CTA: forwards K
constexpr int kScaleWarp = kIssueWarp + 1;          // warp 17: the tiles' scales
// warp 18: odd CTA: forwards V
constexpr int kQueryWarp = kIssueWarp + 3;          // warp 19: copies the queries in; odd CTA: forwards them
constexpr int kPreThreads = 32 * (kQueryWarp + 1);
// Registers a thread, of the 96 each is launched with (65536 / 640): in units
// of a warp's, 8 x 112 + 8 x 96 + 4 x 64 = 20 x 96.  (A thread spills 24 bytes in the
// single CTAs' kernel, 32 in the pairs'.)
constexpr int kSoftRegs = 112, kConvRegs = 96, kMiscRegs = 64;
static_assert(8 * kSoftRegs + 8 * kConvRegs + 4 * kMiscRegs <= 20 * 96, "register split: above it the increase waits forever");
static_assert(kSoftRegs >= 96 && kConvRegs <= 96 && kMiscRegs <= 96, "an increase and two decreases from the launch's 96");

// Shared memory from its base, which is 1024-byte aligned (checked).  The total
// stays under 195 KB: the SM then keeps 60 KB of its 256 KB as L1, where the
// converters' loads in flight live.
constexpr int kStageBytes = 32768;
constexpr int kSmQ = 0;                             // 4 regions [128 rows][64 dims]
constexpr int kSmK = 65536;                         // a pair: 2 stages x 4 regions [64 keys][64 dims]; one CTA: 4 regions [128][64]
constexpr int kSmV = kSmK + 2 * kStageBytes;        // a pair: 2 stages x 2 regions [128 keys][64 dims]; one CTA: 2 x 4 regions [64][64]
constexpr int kSmScale = kSmV + 2 * kStageBytes;    // [2] x {K scales 128, V scales 128, valid blocks, exponent, tile}
constexpr int kScaleSlot = 2 * 512 + 16;
constexpr int kSmRow = kSmScale + 2 * kScaleSlot;   // [2][128] int8 exponents of the rows' factors, by segment parity
constexpr int kSmBar = kSmRow + 2 * kRows;
// Barriers, at the same offsets in both CTAs; [2]: by tile parity.  "Even": the
// issuer waits on the even CTA's, which counts both CTAs' arrivals.  "Both":
// a commit arrives in both CTAs.  A parity wait tells a phase only from the one
// before it; every wait below comes when the phase before is known to be over.
enum : int {
  B_KF = 0,    // [2] even: a tile's K is written (four warps, and the odd CTA's forward); one CTA: [2] its halves
  B_VF = 2,    // [2] even: its V
  B_KL = 4,    // [2] odd: its own half of K, V (four warps), to be forwarded
  B_VL = 6,    // [2]
  B_KE = B_KL, // [2] one CTA alone: Q K^T of half of a tile's dims is done; its K is free
  B_VE = B_VL, // [2] one CTA alone: P V of half of a tile's keys is done; its V is free
  B_SF = 8,    // [2] both: scores of a tile in TMEM; its K stage is free
  B_PF = 10,   // [2] even: P' of a tile in TMEM (every softmax warp of both)
  B_OD = 12,   // [2] both: P V of a tile is done; its V stage is free
  B_SCF = 14,  // [2] scales written (own CTA)
  B_SCE = 16,  // [2] scales read
  B_QF = 18,   // even: queries written
  B_QL = 19,   // odd: its own queries, to be forwarded
  B_QE = 20,   // both: a segment's last Q K^T is done
  B_OE = 21,   // even: a segment's O is read (every softmax warp of both)
  B_RAW = 22,  // the segment's raw queries are read (converter warps)
  B_RAWF = 23, // the segment's raw queries have landed
  B_HELP = 24, // the softmax warps' rows of the first segment's queries are written
  B_DRAIN = 25,
  B_TMEM = 26, // one CTA alone: its tensor memory is allocated
  kPreBars = 27
};
constexpr int kSmTmem = kSmBar + kPreBars * 8;
constexpr int kPreSmem = kSmTmem + 16;
static_assert(kPreSmem <= 195 * 1024, "shared memory");
constexpr uint32_t kTmemO = 0, kTmemS = 256;        // O [0, 256), S of even / odd tiles [256, 384) / [384, 512)

// The B operand of O = P V: V as [key][64 dims] rows of 128 bytes with the
// 128-byte swizzle, dims (N) contiguous: 8-key atoms of 1024 bytes along K,
// regions of the stage's keys (a tile's, or half of one CTA's) x 128 bytes along N.
template <int kN>
__device__ __forceinline__ uint64_t sdesc_v(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kN * 8192 >> 4) << 16;  // leading byte offset: the next 64 dims
  d |= static_cast<uint64_t>(1024 >> 4) << 32;       // stride byte offset: the next 8 keys
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
template <int kN>
constexpr uint32_t kIdescQK = idesc_f16(kN * 128, kTileKeys, false, false);
template <int kN>
constexpr uint32_t kIdescPV = idesc_f16(kN * 128, 256, false, false) | (1u << 16);  // B is N-major

// A run of tiles of one group: a pair's work is one or more of these.
struct Segment {
  int j, g, rg;     // group number (head-major), kv head, row group
  ShGroup grp;
  int t0, t1;       // tiles of the group
  int row0, rows;   // this CTA's first row (of the kv head's n_seq G) and how many there are
};
template <int kN>
__device__ __forceinline__ Segment segment_at(const SharedParams& p, const SharedSeqs& tab, int rank, int x, int x_end) {
  Segment s;
  s.g = x / p.tiles_head;
  const int xh = x - s.g * p.tiles_head;
  s.rg = 0;
  while (s.rg + 1 < p.n_grp && tab.grp[s.rg + 1].x0 <= xh) ++s.rg;
  s.j = s.g * p.n_grp + s.rg;
  s.grp = tab.grp[s.rg];
  s.t0 = xh - s.grp.x0;
  s.t1 = min((s.grp.n_blk + kTileBlocks - 1) / kTileBlocks, s.t0 + (x_end - x));
  s.row0 = s.rg * (kN * kRows) + rank * kRows;
  s.rows = max(0, min(kRows, p.n_seq * p.G - s.row0));
  return s;
}
// Logical block of the b-th visible block of a group.
__device__ __forceinline__ int group_block(const ShGroup& g, int b) { return b < g.sink ? b : g.lo + (b - g.sink); }
// Pool page of it, -1 past the list or outside the pool.
__device__ __forceinline__ int group_page(const SharedParams& p, const ShGroup& g, int b) {
  if (b >= g.n_blk) return -1;
  const int phys = __ldg(p.block_table + group_block(g, b));
  return phys >= 0 && phys < p.n_pool ? phys : -1;
}

struct PreCtx {
  uint32_t sb;    // shared base, the same offset in both CTAs
  uint32_t tm;    // TMEM base, the same in both
  int rank;       // 0: the even CTA of the pair, 1: the odd one
  int x0, x1;     // the pair's tiles
  WaitCtl wc;
  __device__ uint32_t bar(int i) const { return sb + kSmBar + 8 * i; }
  // One outcome for the warp.
  __device__ bool wait(int i, uint32_t parity) const {
    return __all_sync(kAllLanes, mbar_wait(bar(i), parity & 1u, wc, 80 + i));
  }
  // As wait, for a phase that takes as many tiles as a segment has (131072 keys:
  // 1024 tiles, 1.7 ms): the limit starts again whenever the scale warp, at most
  // two tiles ahead of the softmax, has written another pair of tiles' scales.
  __device__ bool wait_while_tiles_go_on(int i, uint32_t parity) const {
    auto tile = [&] {
      uint32_t n;
      asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(n) : "r"(sb + kSmScale + 1024 + 8));
      return n;
    };
    uint32_t seen = tile();
    uint64_t t0 = globaltimer_ns();
    bool ok = false;
    for (uint32_t k = 1; !(ok = mbar_try_wait_sleep(bar(i), parity & 1u, 20000u)); ++k) {
      if (k & 31u) continue;
      if (*reinterpret_cast<volatile int*>(wc.err) != 0) break;
      const uint32_t now = tile();
      if (now != seen) {
        seen = now;
        t0 = globaltimer_ns();
      } else if (globaltimer_ns() - t0 > wc.limit_ns) {
        atomicCAS(wc.err, 0, DEV_ERR_TIMEOUT | ((80 + i) & 0xff));
        break;
      }
    }
    return __all_sync(kAllLanes, ok);
  }
  // An arrival on the even CTA's barrier that hands over tensor memory (the
  // caller has waited for its tcgen05 accesses and fenced them).
  __device__ void arrive_even_tmem(int i) const {
    if (rank == 0) mbar_arrive(bar(i));
    else mbar_arrive_remote(cluster_addr(bar(i), 0));
  }
};

// ---- converters.  A warp keeps its share of a tile's codes in registers, 16
// bytes x 8 a thread: it widens what has arrived into the stage of the tile's
// parity and then loads its part of the next tile.
// 16 codes of one row as 32 bytes: pieces 2 (u % 4) and + 1 of a 128-byte
// swizzled row.  Of the eight threads whose stores go together four have an
// even and four the next, odd row, whose pieces are swizzled to odd places:
// eight different ones.
__device__ __forceinline__ void widen16(const uint4 c, uint32_t row_addr, int row, int u) {
  const uint32_t w[4] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u, c.z ^ 0x80808080u, c.w ^ 0x80808080u};
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[2 * e] = lo_pair(w[e]), h[2 * e + 1] = hi_pair(w[e]);
  const uint32_t at = row_addr + (uint32_t)(((2 * (u & 3)) ^ (row & 7)) << 4);
  sts128(at, h[0], h[1], h[2], h[3]);
  sts128(at ^ 16u, h[4], h[5], h[6], h[7]);
}

// ---- queries.  Rows [first, end) of the CTA's, from their raw copies: each row
// scaled by a power of two and rounded to fp16, exactly.  Four rows at a time,
// their chains of shuffles side by side; a row's largest magnitude from the bf16
// bit patterns, two rows to a word.
__device__ __forceinline__ void stage_queries(const PreCtx& c, const Segment& s, uint32_t raw, uint32_t rowc, int first, int end) {
  const int lane = threadIdx.x & 31;
  const int last = max(0, s.rows - 1);  // rows past the last hold anything: no one reads their results
#pragma unroll 1
  for (int i0 = first; i0 < end; i0 += 4) {
    uint4 q[4];
    uint32_t m[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[i] = lds_u32x4(raw + min(i0 + i, last) * (kHeadDim * 2) + 16 * lane);
      uint32_t a = __vmaxu2(__vmaxu2(q[i].x & 0x7fff7fffu, q[i].y & 0x7fff7fffu), __vmaxu2(q[i].z & 0x7fff7fffu, q[i].w & 0x7fff7fffu));
      a = max(a & 0xffffu, a >> 16);
      m[i >> 1] = i & 1 ? m[i >> 1] | a << 16 : a;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < 2; ++i) m[i] = __vmaxu2(m[i], __shfl_xor_sync(kAllLanes, m[i], o));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i0 + i;
      const int k = row_shift(__uint_as_float(i & 1 ? m[i >> 1] & 0xffff0000u : m[i >> 1] << 16));
      const float mul = pow2i(k);
      const uint32_t u[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = mul2(make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u)), make_float2(mul, mul));
        h[e] = pack_f16x2(v.x, v.y);
      }
      sts128(c.sb + kSmQ + (lane >> 3) * 16384 + row * 128 + (((lane & 7) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
      if (lane == 0) asm volatile("st.shared.u8 [%0], %1;" ::"r"(rowc + row), "r"(-k) : "memory");
    }
  }
  fence_proxy_async_shared();
  __syncwarp();
}
// The first segment's raw rows lie in the V stages, the others' in the K stages:
// the first ones' staging, by the idle softmax warps and the V warps, then runs
// beside the widening of the first K tile, while a later segment's must not wait
// for the last P V of the one before.
constexpr int kHelpRows = 12;  // each softmax warp's; the four V warps share the others
static_assert(kSoftWarps * kHelpRows + 4 * 8 == kRows, "rows of the first segment");
template <int kN>
__device__ __forceinline__ bool help_stage(const SharedParams& p, const SharedSeqs& tab, const PreCtx& c) {
  const int warp = threadIdx.x >> 5;
  const Segment s = segment_at<kN>(p, tab, c.rank, c.x0, c.x1);
  if (!c.wait(B_RAWF, 0)) return false;
  stage_queries(c, s, c.sb + kSmV, c.sb + kSmRow, kHelpRows * warp, kHelpRows * (warp + 1));
  if ((threadIdx.x & 31) == 0) mbar_arrive(c.bar(B_HELP));
  return true;
}

// One code for K and V warps: the kernel's instructions exceed the caches that
// feed the schedulers, and every line of it is fetched anew for each tile.
template <int kN>
__device__ __forceinline__ void role_convert(const SharedParams& p, const SharedSeqs& tab, const PreCtx& c) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - kSoftWarps;
  const bool kv = warp >= kConvWarps / 2;  // V
  const int w = warp & 3;
  uint32_t n_step = 0, n_seg = 0;  // steps: a pair's tiles, one CTA's parts of tiles
  const size_t tok = (size_t)p.HKV * kHeadDim;  // bytes from a token to the next
  // What a warp widens at a time lies in one of two places of 32 KB:
  //   a pair's K: keys 64 rank + 16 w on, all dims; one CTA's V: 64 of the tile's
  //   keys (part h), of them 16 w on, all dims.  A load takes two keys.
  //   wide: a pair's V: keys 32 w on, dims 128 rank on; one CTA's K: keys 32 w on,
  //   dims 128 h on.  A load takes four keys.
  // Lane bit 2 (and 4) the key, the others the 16 bytes.
  const bool wide = kv == (kN == 2);
  const int u = wide ? (lane & 3) | (lane >> 1 & 4) : (lane & 3) | (lane >> 3) << 2;
  const int sub = wide ? (lane >> 2 & 1) | (lane >> 4) << 1 : lane >> 2 & 1;
  const int step = wide ? 4 : 2;                                // keys per load
  const int row0 = (wide ? 32 : 16) * w + sub;                  // the place's row of the lane's first load
  const uint32_t at0 = c.sb + (kv ? kSmV : kSmK) + (u >> 2) * (wide ? 16384 : 8192) + row0 * 128;
  const int blk0 = wide ? 2 * w : 4 * c.rank + w;               // first block of the tile it loads
  const size_t step_b = step * tok, half_b = wide ? 0 : 8 * tok;  // from a load to the next; from load 0 to load 4
  const int blk4 = wide ? blk0 + 1 : blk0;                      // block of load 4
  const int8_t* base = (kv ? p.v_pool + (wide ? 128 * c.rank : 0) : p.k_pool) + 16 * u + (size_t)sub * tok;
  constexpr int kParts = 2 / kN;
  for (int x = c.x0; x < c.x1; ++n_seg) {
    const Segment s = segment_at<kN>(p, tab, c.rank, x, c.x1);
    const int8_t* src = base + (size_t)s.g * kHeadDim;
    // pages of the segment's blocks, 32 at a time, one per lane
    const int b0 = s.t0 * kTileBlocks;
    int pg = group_page(p, s.grp, b0 + lane), pg_next = group_page(p, s.grp, b0 + 32 + lane);
    uint4 r[8];
    // a block past the list or of a bad page loads page 0's codes: whatever finite values they widen to,
    // the softmax gives those keys no weight
    auto load = [&](int t4, int h) {
      const int more = kN == 1 && kv ? 4 * h : 0;  // blocks
      const int pa = max(0, __shfl_sync(kAllLanes, pg, t4 * kTileBlocks + blk0 + more));
      const int pb = max(0, __shfl_sync(kAllLanes, pg, t4 * kTileBlocks + blk4 + more));
      const int8_t* part = src + (kN == 1 && !kv ? 128 * h : 0);
      const int8_t* a = part + (size_t)pa * (kPage * tok);
      const int8_t* b = part + (size_t)pb * (kPage * tok) + half_b;
#pragma unroll
      for (int n = 0; n < 4; ++n, a += step_b) r[n] = ldg_stream(a);
#pragma unroll
      for (int n = 4; n < 8; ++n, b += step_b) r[n] = ldg_stream(b);
    };
    load(0, 0);
    if (n_seg > 0 || kv) {
      if (!c.wait(B_RAWF, n_seg)) return;
      const int first = n_seg > 0 ? 16 * warp : kSoftWarps * kHelpRows + 8 * w;
      stage_queries(c, s, c.sb + (n_seg > 0 ? kSmK : kSmV), c.sb + kSmRow + (n_seg & 1) * kRows, first,
                    first + (n_seg > 0 ? 16 : 8));
      if (n_seg == 0 && !c.wait(B_HELP, 0)) return;
    }
    if (lane == 0) {
      mbar_arrive(c.bar(B_RAW));
      mbar_arrive(c.bar(c.rank == 0 ? B_QF : B_QL));
    }
    // every warp has read its raw rows: the stages that held them may be written
    if ((n_seg > 0 || kv) && !c.wait(B_RAW, n_seg)) return;

    const int steps = (s.t1 - s.t0) * kParts;
    for (int i = 0; i < steps; ++i, ++n_step) {
      const int t_next = (i + 1) / kParts, h_next = (i + 1) % kParts;  // what is loaded next
      if (h_next == 0 && (t_next & 3) == 0) {  // its pages are in the next window
        pg = pg_next;
        pg_next = group_page(p, s.grp, b0 + 8 * t_next + 32 + lane);
      }
      // the products that read what was in this place are done
      const uint32_t st = n_step & 1;
      if (n_step > 1 && !c.wait((kv ? (kN == 2 ? B_OD : B_VE) : (kN == 2 ? B_SF : B_KE)) + st, (n_step >> 1) - 1)) return;
#pragma unroll
      for (int n = 0; n < 8; ++n) widen16(r[n], at0 + st * kStageBytes + step * n * 128, row0 + step * n, u);
      fence_proxy_async_shared();
      __syncwarp();
      // K warps take no part in the first segment's staging; they see that its
      // rows have landed all the same, before their first tile leads to the next
      // segment's: a parity wait there would take this phase's for it.
      if (n_step == 0 && !kv && !c.wait(B_RAWF, 0)) return;
      if (lane == 0) mbar_arrive(c.bar((kv ? (c.rank == 0 ? B_VF : B_VL) : (c.rank == 0 ? B_KF : B_KL)) + st));
      if (i + 1 < steps) load(t_next & 3, h_next);
    }
    x += s.t1 - s.t0;
  }
}

// ---- forwards of the odd CTA: the even CTA's issuer learns that the odd CTA's
// part of a tile (of a segment's queries) is written.  A cluster-scope release
// takes ~1100 cycles, so it has a thread of its own.
__device__ __forceinline__ void role_forward_tiles(const PreCtx& c, int local, int even) {
  for (int n = 0; n < c.x1 - c.x0; ++n) {
    if (!mbar_wait(c.bar(local + (n & 1)), (n >> 1) & 1, c.wc, 80 + local)) return;
    mbar_arrive_cluster(cluster_addr(c.bar(even + (n & 1)), 0));
  }
}
// The segments' query rows, copied as they are (into the K stages: free, the
// segment before's last Q K^T is done): the G rows of a sequence lie together.
__device__ __forceinline__ void copy_queries(const SharedParams& p, const SharedSeqs& tab, const PreCtx& c, const Segment& s,
                                             uint32_t raw) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) mbar_expect_tx(c.bar(B_RAWF), s.rows * (kHeadDim * 2));
  __syncwarp();
  const int n = s.rows >> p.log2_g, s0 = s.row0 >> p.log2_g;  // whole sequences: 128 is a multiple of G
  for (int i = lane; i < n; i += 32)
    bulk_load(raw + i * p.G * (kHeadDim * 2), p.q + ((size_t)tab.s[s0 + i].x * p.HQ + (size_t)s.g * p.G) * kHeadDim,
              p.G * (kHeadDim * 2), c.bar(B_RAWF));
}
// The first segment's copies have been issued.  In the odd CTA also the forward
// of its queries.
template <int kN>
__device__ __forceinline__ void role_queries(const SharedParams& p, const SharedSeqs& tab, const PreCtx& c) {
  const int lane = threadIdx.x & 31;
  uint32_t n_seg = 0, copied = 1;
  for (int x = c.x0; x < c.x1; ++n_seg) {
    const Segment s = segment_at<kN>(p, tab, c.rank, x, c.x1);
    if (n_seg > 0) {
      if (!c.wait_while_tiles_go_on(B_QE, n_seg - 1)) break;
      copy_queries(p, tab, c, s, c.sb + kSmK);
      ++copied;
    }
    if (c.rank == 1) {
      if (!c.wait(B_QL, n_seg)) break;
      if (lane == 0) mbar_arrive_cluster(cluster_addr(c.bar(B_QF), 0));
    }
    x += s.t1 - s.t0;
  }
  // no copy is in flight when the CTA leaves, whatever gave up
  (void)mbar_wait_drain(c.bar(B_RAWF), (copied - 1) & 1u, kShDrainNs);
  __syncwarp();
}

// ---- scales of every tile's keys, V's normalised by a running power of two.
template <int kN>
__device__ __forceinline__ void role_scales(const SharedParams& p, const SharedSeqs& tab, const PreCtx& c) {
  const int lane = threadIdx.x & 31;
  uint32_t n_tile = 0;
  for (int x = c.x0; x < c.x1;) {
    const Segment s = segment_at<kN>(p, tab, c.rank, x, c.x1);
    int ev = -100;
    // lane: keys 4 lane .. + 3 of a tile, in block lane / 4
    float ks[4], vs[4];
    bool valid = false;
    auto load = [&](int t) {
      const int b = t * kTileBlocks + (lane >> 2);
      const int page = group_page(p, s.grp, b);
      valid = page >= 0;
      if (!valid && b < s.grp.n_blk && (lane & 3) == 0) record_bad_page(p.err);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const size_t at = ((size_t)(valid ? page : 0) * kPage + 4 * (lane & 3) + e) * p.HKV + s.g;
        ks[e] = valid ? __ldg(p.k_scale + at) : 0.f;
        vs[e] = valid ? __ldg(p.v_scale + at) : 0.f;
      }
    };
    load(s.t0);
    for (int t = s.t0; t < s.t1; ++t, ++n_tile) {
      const int b = n_tile & 1;
      float mv = fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mv = fmaxf(mv, __shfl_xor_sync(kAllLanes, mv, o));
      ev = max(ev, exp_above(mv));
      const float vn = pow2i(-ev);
      const uint32_t ok = __ballot_sync(kAllLanes, valid);
      if (n_tile > 1 && !c.wait(B_SCE + b, (n_tile >> 1) - 1)) return;
      const uint32_t at = c.sb + kSmScale + b * kScaleSlot;
      sts128(at + 16 * lane, __float_as_uint(ks[0]), __float_as_uint(ks[1]), __float_as_uint(ks[2]), __float_as_uint(ks[3]));
      sts128(at + 512 + 16 * lane, __float_as_uint(vs[0] * vn), __float_as_uint(vs[1] * vn), __float_as_uint(vs[2] * vn),
             __float_as_uint(vs[3] * vn));
      if (lane == 0) {
        uint32_t m8 = 0;
#pragma unroll
        for (int e = 0; e < kTileBlocks; ++e) m8 |= ((ok >> (4 * e)) & 1u) << e;
        sts128(at + 1024, m8, (uint32_t)ev, n_tile, 0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar(B_SCF + b));
      if (t + 1 < s.t1) load(t + 1);
    }
    x += s.t1 - s.t0;
  }
}

// ---- the products, one thread (of a pair's even CTA).  A tile's instructions go out
// of one asm block with the operands' offsets added inside it: instructions
// between them, a branch above all, leave the tensor pipe waiting.
// S = Q K^T: four regions of 64 dims, four k-steps of 32 bytes each.
#define PA_SH_QK(G, qo, ko)                                \
  "add.s64 a, %1, " qo ";\n\tadd.s64 b, %2, " ko ";\n\t" \
  "tcgen05.mma.cta_group::" G ".kind::f16 [%0], a, b, %3, pt;\n\t"
#define PA_SH_QK4(G, r, K)                                                                            \
  PA_SH_QK(G, r " * 1024", r " * " K) PA_SH_QK(G, r " * 1024 + 2", r " * " K " + 2")                  \
      PA_SH_QK(G, r " * 1024 + 4", r " * " K " + 4") PA_SH_QK(G, r " * 1024 + 6", r " * " K " + 6")
#define PA_SH_QK_FIRST(G)                                                                             \
  "{\n\t.reg .pred p0, pt;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p0, %4, 0;\n\tsetp.eq.b32 pt, %4, %4;\n\t" \
  "tcgen05.mma.cta_group::" G ".kind::f16 [%0], %1, %2, %3, p0;\n\t"                                  \
  PA_SH_QK(G, "2", "2") PA_SH_QK(G, "4", "4") PA_SH_QK(G, "6", "6")
// A pair: the whole tile, each CTA with its 64 keys of K.
__device__ __forceinline__ void mma_qk_pair(uint32_t d, uint64_t qd, uint64_t kd) {
  asm volatile(PA_SH_QK_FIRST("2") PA_SH_QK4("2", "1", "512") PA_SH_QK4("2", "2", "512") PA_SH_QK4("2", "3", "512") "}" ::"r"(d),
               "l"(qd), "l"(kd), "r"(kIdescQK<2>), "r"(0u) : "memory");
}
// One CTA: half of the dims of 128 keys.
__device__ __forceinline__ void mma_qk_half(uint32_t d, uint64_t qd, uint64_t kd, uint32_t acc0) {
  asm volatile(PA_SH_QK_FIRST("1") PA_SH_QK4("1", "1", "1024") "}" ::"r"(d), "l"(qd), "l"(kd), "r"(kIdescQK<1>), "r"(acc0)
               : "memory");
}
// O (+)= P V over a stage's keys: k-steps of 16 keys, 8 TMEM columns of P' and 2048 bytes of V each.
#define PA_SH_PV(G, po, vo)                                \
  "add.u32 a, %1, " po ";\n\tadd.s64 b, %2, " vo ";\n\t" \
  "tcgen05.mma.cta_group::" G ".kind::f16 [%0], [a], b, %3, pt;\n\t"
#define PA_SH_PV_FIRST(G)                                                                                         \
  "{\n\t.reg .pred p0, pt;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\tsetp.ne.b32 p0, %4, 0;\n\tsetp.eq.b32 pt, %4, %4;\n\t" \
  "tcgen05.mma.cta_group::" G ".kind::f16 [%0], [%1], %2, %3, p0;\n\t"                                            \
  PA_SH_PV(G, "8", "128") PA_SH_PV(G, "16", "256") PA_SH_PV(G, "24", "384")
template <int kN>
__device__ __forceinline__ void mma_pv_tile(uint32_t d, uint32_t ptm, uint64_t vd, uint32_t acc0) {
  if constexpr (kN == 2)
    asm volatile(PA_SH_PV_FIRST("2") PA_SH_PV("2", "32", "512") PA_SH_PV("2", "40", "640") PA_SH_PV("2", "48", "768")
                 PA_SH_PV("2", "56", "896") "}" ::"r"(d), "r"(ptm), "l"(vd), "r"(kIdescPV<2>), "r"(acc0) : "memory");
  else
    asm volatile(PA_SH_PV_FIRST("1") "}" ::"r"(d), "r"(ptm), "l"(vd), "r"(kIdescPV<1>), "r"(acc0) : "memory");
}
static_assert((16384 >> 4) == 1024 && (8192 >> 4) == 512 && (2048 >> 4) == 128, "descriptor steps of the blocks above");
template <int kN>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (kN == 2) mma_commit_pair(bar);
  else mma_commit(bar);
}

// Q K^T of tile t + 1 goes before P V of tile t, so that the tensor core has
// the next scores to compute while the softmax handles these.  The parity waits:
// a tile's K, V, P' and queries are written only after the products that read
// what was there before.
template <int kN>
__device__ __forceinline__ void role_issue(const SharedParams& p, const SharedSeqs& tab, const PreCtx& c) {
  uint32_t n_tile = 0, n_seg = 0;
  bool ok = true;
  const uint64_t qd = sdesc_k_sw128(c.sb + kSmQ);
  const uint64_t kd0 = sdesc_k_sw128(c.sb + kSmK), kd1 = sdesc_k_sw128(c.sb + kSmK + kStageBytes);
  const uint64_t vd0 = sdesc_v<kN>(c.sb + kSmV), vd1 = sdesc_v<kN>(c.sb + kSmV + kStageBytes);
  // K, V and queries of the odd CTA come with a cluster-scope release
  auto wait_pair = [&](int i, uint32_t parity) {
    return kN == 2 ? mbar_wait_cluster(c.bar(i), parity & 1u, c.wc, 80 + i) : mbar_wait(c.bar(i), parity & 1u, c.wc, 80 + i);
  };
  auto wait = [&](int i, uint32_t parity) { return mbar_wait(c.bar(i), parity & 1u, c.wc, 80 + i); };
  auto qk = [&](uint32_t n) {  // n: the tile's number in the unit's order
    const uint32_t d = c.tm + kTmemS + 128 * (n & 1);
    if (kN == 2) {
      if (!wait_pair(B_KF + (n & 1), n >> 1)) return false;
      tc_fence_after();
      mma_qk_pair(d, qd, (n & 1) ? kd1 : kd0);
    } else {
      if (!wait(B_KF, n)) return false;
      tc_fence_after();
      mma_qk_half(d, qd, kd0, 0);
      commit<kN>(c.bar(B_KE));
      if (!wait(B_KF + 1, n)) return false;
      tc_fence_after();
      mma_qk_half(d, qd + 2048, kd1, 1);
      commit<kN>(c.bar(B_KE + 1));
    }
    commit<kN>(c.bar(B_SF + (n & 1)));
    return true;
  };
  auto pv = [&](uint32_t n, uint32_t acc) {
    const uint32_t ptm = c.tm + kTmemS + 128 * (n & 1);
    if (kN == 2) {
      if (!wait_pair(B_VF + (n & 1), n >> 1) || !wait(B_PF + (n & 1), n >> 1)) return false;
      tc_fence_after();
      mma_pv_tile<kN>(c.tm + kTmemO, ptm, (n & 1) ? vd1 : vd0, acc);
    } else {
      if (!wait(B_PF + (n & 1), n >> 1) || !wait(B_VF, n)) return false;
      tc_fence_after();
      mma_pv_tile<kN>(c.tm + kTmemO, ptm, vd0, acc);
      commit<kN>(c.bar(B_VE));
      if (!wait(B_VF + 1, n)) return false;
      tc_fence_after();
      mma_pv_tile<kN>(c.tm + kTmemO, ptm + 32, vd1, 1);
      commit<kN>(c.bar(B_VE + 1));
    }
    commit<kN>(c.bar(B_OD + (n & 1)));
    return true;
  };
  for (int x = c.x0; ok && x < c.x1; ++n_seg) {
    const Segment s = segment_at<kN>(p, tab, c.rank, x, c.x1);
    const int nt = s.t1 - s.t0;
    ok = wait_pair(B_QF, n_seg) && qk(n_tile);
    if (nt == 1) commit<kN>(c.bar(B_QE));
    // the epilogue has read the segment before's O
    ok = ok && (n_seg == 0 || wait(B_OE, n_seg - 1));
    for (int t = 1; ok && t < nt; ++t) {
      ok = qk(n_tile + t);
      if (t == nt - 1) commit<kN>(c.bar(B_QE));
      ok = ok && pv(n_tile + t - 1, t > 1);
    }
    ok = ok && pv(n_tile + nt - 1, nt > 1);
    n_tile += nt;
    x += nt;
  }
  // nothing may be in flight when the CTAs free their TMEM
  commit<kN>(c.bar(B_DRAIN));
  (void)mbar_wait_drain(c.bar(B_DRAIN), 0, kShDrainNs);
}

// ---- softmax.  A warp owns 16 rows, read in the 16-lane TMEM shape: a thread
// holds rows t / 4 and t / 4 + 8 and, of every eight keys, keys 2 (t % 4) and
// + 1, so that each scale it loads from shared memory serves two rows.
struct SliceRows {
  float c[2], m[2];  // the rows' factors, their references in log2 units
  float2 l[2];       // their sums, this thread's keys
  int win_lo[2];
};

// z = score * k_scale, and the rows' maxima.
template <bool kMasked>
__device__ __forceinline__ void scale_and_max(uint32_t (&s)[64], uint32_t ks_at, uint32_t seen0, uint32_t seen1,
                                              float& z0, float& z1) {
  float za = -INFINITY, zb = -INFINITY;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    float2 ks;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks.x), "=f"(ks.y) : "r"(ks_at + 32 * k));
    float2 a = mul2(make_float2(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1])), ks);
    float2 b = mul2(make_float2(__uint_as_float(s[4 * k + 2]), __uint_as_float(s[4 * k + 3])), ks);
    if (kMasked) {
      if (!(seen0 >> (k >> 1) & 1u)) a = make_float2(-INFINITY, -INFINITY);
      if (!(seen1 >> (k >> 1) & 1u)) b = make_float2(-INFINITY, -INFINITY);
    }
    s[4 * k] = __float_as_uint(a.x);
    s[4 * k + 1] = __float_as_uint(a.y);
    s[4 * k + 2] = __float_as_uint(b.x);
    s[4 * k + 3] = __float_as_uint(b.y);
    za = max3(za, a.x, a.y);
    zb = max3(zb, b.x, b.y);
  }
  z0 = za;
  z1 = zb;
}

// One tile of the warp's rows: P' over its scores.  `first`: no O to rescale yet.
__device__ __forceinline__ bool softmax_tile(const SharedParams& p, const PreCtx& c, const ShGroup& grp, int blk0,
                                             uint32_t stm, uint32_t otm, uint32_t sc, uint32_t valid, float fe,
                                             bool first, uint32_t n_before, SliceRows& r) {
  const int lane = threadIdx.x & 31;
  const uint32_t ks_at = sc + 8 * (lane & 3);
  uint32_t s[64];
  tmem_ld_16x256b_x16(stm, s);
  uint32_t seen[2] = {valid, valid};  // blocks of the tile that the rows see
  if (p.W > 0) {
#pragma unroll
    for (int e = 0; e < kTileBlocks; ++e) {
      const int lb = group_block(grp, blk0 + e);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (lb >= p.S && lb < r.win_lo[i]) seen[i] &= ~(1u << e);
    }
  }
  tmem_wait_ld(s);
  float z[2];
  if (__all_sync(kAllLanes, (seen[0] & seen[1]) == 0xffu)) scale_and_max<false>(s, ks_at, 0, 0, z[0], z[1]);
  else scale_and_max<true>(s, ks_at, seen[0], seen[1], z[0], z[1]);
  // The rows' references.  Mostly no row passes its own by enough to move it,
  // which each thread sees from its own keys; only else are the rows' maxima
  // put together.
  float f[2] = {fe, fe};  // what earlier P V shrink by
  bool need = false;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    need |= z[i] != -INFINITY && (r.m[i] == -INFINITY || z[i] * r.c[i] > r.m[i] + kMaxLift);
  need = __any_sync(kAllLanes, need);
  if (need) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      z[i] = fmaxf(z[i], __shfl_xor_sync(kAllLanes, z[i], 1));
      z[i] = fmaxf(z[i], __shfl_xor_sync(kAllLanes, z[i], 2));
      const float mz = z[i] == -INFINITY ? -INFINITY : z[i] * r.c[i];
      if (r.m[i] == -INFINITY) {  // sums and products so far are zero
        r.m[i] = mz;
      } else if (mz > r.m[i] + kMaxLift) {
        const float g = ex2f(r.m[i] - mz);
        r.m[i] = mz;
        r.l[i] = mul2(r.l[i], make_float2(g, g));
        f[i] *= g;
      }
    }
  }
  // p = 2^(z c - m), P' = p v_scale 2^-ev in fp16.  A hidden key's z is -inf,
  // and a row's factor may be 0: keep the product -inf.
  const float n0 = r.m[0] == -INFINITY ? 0.f : -r.m[0], n1 = r.m[1] == -INFINITY ? 0.f : -r.m[1];
  const float c0 = fmaxf(r.c[0], 1e-30f), c1 = fmaxf(r.c[1], 1e-30f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // 64 keys
    uint32_t ph[16];
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const int k = 8 * h + kk;
      float2 vs;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(vs.x), "=f"(vs.y) : "r"(ks_at + 512 + 32 * k));
      const float2 ya = fma2(make_float2(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1])), make_float2(c0, c0), make_float2(n0, n0));
      const float2 yb = fma2(make_float2(__uint_as_float(s[4 * k + 2]), __uint_as_float(s[4 * k + 3])), make_float2(c1, c1), make_float2(n1, n1));
      const float2 ea = make_float2(ex2f(ya.x), ex2f(ya.y)), eb = make_float2(ex2f(yb.x), ex2f(yb.y));
      r.l[0] = add2(r.l[0], ea);
      r.l[1] = add2(r.l[1], eb);
      const float2 wa = mul2(ea, vs), wb = mul2(eb, vs);
      ph[2 * kk] = pack_f16x2(wa.x, wa.y);
      ph[2 * kk + 1] = pack_f16x2(wb.x, wb.y);
    }
    tmem_st_16x128b_x8(stm + 32 * h, ph);
  }
  // O takes the same factors; last, when the scores' registers are free for it
  if (!first && (fe != 1.f || (need && __any_sync(kAllLanes, f[0] != 1.f || f[1] != 1.f)))) {
    // P V of the tile before (that of two tiles before came ahead of this tile's scores)
    if (!c.wait(B_OD + (n_before & 1), n_before >> 1)) return false;
    tc_fence_after();
    uint32_t o[64];  // 128 columns
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      tmem_ld_16x256b_x16(otm + 128 * h, o);
      tmem_wait_ld(o);
#pragma unroll
      for (int e = 0; e < 64; e += 4) {
        const float2 a = mul2(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), make_float2(f[0], f[0]));
        const float2 b = mul2(make_float2(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])), make_float2(f[1], f[1]));
        o[e] = __float_as_uint(a.x);
        o[e + 1] = __float_as_uint(a.y);
        o[e + 2] = __float_as_uint(b.x);
        o[e + 3] = __float_as_uint(b.y);
      }
      tmem_st_16x256b_x16(otm + 128 * h, o);
    }
  }
  return true;
}

template <int kN>
__device__ __forceinline__ void role_softmax(const SharedParams& p, const SharedSeqs& tab, const PreCtx& c) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = 32 * (warp & 3), half = warp >> 2;
  const uint32_t lanes = (uint32_t)(quad + 16 * half) << 16;  // the warp's 16 rows
  const int row0 = quad + 16 * half + (lane >> 2);            // this thread's: row0, row0 + 8
  uint32_t n_tile = 0, n_seg = 0;
  for (int x = c.x0; x < c.x1; ++n_seg) {
    const Segment s = segment_at<kN>(p, tab, c.rank, x, c.x1);
    const int nt = s.t1 - s.t0;
    SliceRows r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row0 + 8 * i;
      r.m[i] = -INFINITY;
      r.l[i] = make_float2(0.f, 0.f);
      r.win_lo[i] = p.W > 0 && row < s.rows ? tab.s[(s.row0 + row) >> p.log2_g].w : 0;
    }
    int ev = -100;
    for (int t = 0; t < nt; ++t, ++n_tile) {
      const int b = n_tile & 1;
      const uint32_t stm = c.tm + kTmemS + 128 * b + lanes;
      if (!c.wait(B_SCF + b, n_tile >> 1) || !c.wait(B_SF + b, n_tile >> 1)) return;
      tc_fence_after();
      if (t == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          int e;
          asm volatile("ld.shared.s8 %0, [%1];" : "=r"(e) : "r"(c.sb + kSmRow + (n_seg & 1) * kRows + row0 + 8 * i));
          r.c[i] = pow2i(e) * p.sm_scale_log2;
        }
      }
      const uint32_t sc = c.sb + kSmScale + b * kScaleSlot;
      const float4 meta = lds_f32x4(sc + 1024);
      const int ev_t = (int)__float_as_uint(meta.y);
      const float fe = ev_t > ev ? pow2i(max(-126, ev - ev_t)) : 1.f;
      ev = ev_t;
      if (!softmax_tile(p, c, s.grp, (s.t0 + t) * kTileBlocks, stm, c.tm + kTmemO + lanes, sc, __float_as_uint(meta.x), fe,
                        t == 0, n_tile - 1, r))
        return;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        c.arrive_even_tmem(B_PF + b);
        mbar_arrive(c.bar(B_SCE + b));
      }
    }
    // the segment's partial: one row a thread, the quadrant's two warps half of the dims each
    if (!c.wait(B_OD + ((n_tile - 1) & 1), (n_tile - 1) >> 1)) return;
    tc_fence_after();
    const int id = (int)blockIdx.x / kN + s.j, row = quad + lane;
    const float up = pow2i(ev);
    float4* dst = p.pre_o + ((size_t)id * 64 + 32 * half) * (kN * kRows) + c.rank * kRows + row;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {  // 64 columns
      uint32_t o[2][32];
      const uint32_t at = c.tm + kTmemO + 128 * half + 64 * h + ((uint32_t)quad << 16);
      tmem_ld32(at, o[0]);
      tmem_ld32(at + 32, o[1]);
      tmem_wait_ld(o[0]);
      reg_fence(o[1]);
      if (row < s.rows) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t* v = o[e >> 3] + 4 * (e & 7);
          dst[(size_t)(16 * h + e) * (kN * kRows)] =
              make_float4(__uint_as_float(v[0]) * up, __uint_as_float(v[1]) * up, __uint_as_float(v[2]) * up,
                          __uint_as_float(v[3]) * up);
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) c.arrive_even_tmem(B_OE);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = r.l[i].x + r.l[i].y;
      sum += __shfl_xor_sync(kAllLanes, sum, 1);
      sum += __shfl_xor_sync(kAllLanes, sum, 2);
      if ((lane & 3) == 0 && row0 + 8 * i < s.rows)
        p.pre_ml[(size_t)id * (kN * kRows) + c.rank * kRows + row0 + 8 * i] = make_float2(r.m[i], sum);
    }
    x += nt;
  }
}

template <int kN>
__device__ __forceinline__ void prefix_pass(const SharedParams& p, const SharedSeqs& tab) {
  extern __shared__ __align__(1024) uint8_t raw[];
  PreCtx c;
  c.sb = smem_u32(raw);
  if (c.sb & 1023u) {  // every thread of both CTAs: nothing was started
    if (threadIdx.x == 0) atomicCAS(p.err, 0, DEV_ERR_LAYOUT);
    return;
  }
  c.wc = WaitCtl{p.err, p.wait_ns};
  c.rank = kN == 2 ? (int)cluster_rank() : 0;
  c.x0 = tab.cut[blockIdx.x / kN];
  c.x1 = tab.cut[blockIdx.x / kN + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < kPreBars) {
    const int i = threadIdx.x;
    int n = 1;
    if (i < B_KL) n = kConvWarps / 2 + kN - 1;
    if (i >= B_KL && i < B_SF) n = kN == 2 ? kConvWarps / 2 : 1;
    if (i == B_QF) n = kConvWarps + kN - 1;
    if (i == B_QL || i == B_RAW) n = kConvWarps;
    if ((i >= B_SCE && i < B_QF) || i == B_HELP) n = kSoftWarps;
    if ((i >= B_PF && i < B_OD) || i == B_OE) n = kN * kSoftWarps;
    mbar_init(c.bar(i), n);
    fence_mbar_init();
  }
  __syncthreads();
  // The first segment's queries come in and are staged, and its first K tile is
  // widened, while the pair's tensor memory is allocated and the CTAs meet: only
  // what reaches into the other CTA or tensor memory waits for that.
  if (warp == kQueryWarp) copy_queries(p, tab, c, segment_at<kN>(p, tab, c.rank, c.x0, c.x1), c.sb + kSmV);
  if (warp == kIssueWarp) {
    if constexpr (kN == 2) {
      tmem_alloc_pair(c.sb + kSmTmem, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(c.sb + kSmTmem, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (kN == 2) {
    cluster_arrive();
  } else {
    __syncwarp();
    if (warp == kIssueWarp && lane == 0) mbar_arrive(c.bar(B_TMEM));
  }
  dependents_may_start();
  auto meet = [&] {  // both CTAs have their barriers and tensor memory; once in every thread
    bool ok = true;
    if constexpr (kN == 2) cluster_wait();
    else ok = c.wait(B_TMEM, 0);
    tc_fence_after();
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(c.tm) : "r"(c.sb + kSmTmem));
    return ok;
  };
  if (warp < kSoftWarps) {
    more_regs<kSoftRegs>();
    const bool ok = help_stage<kN>(p, tab, c);
    if (meet() && ok) role_softmax<kN>(p, tab, c);
  } else if (warp < kIssueWarp) {
    fewer_regs<kConvRegs>();
    role_convert<kN>(p, tab, c);
    (void)meet();
  } else {
    fewer_regs<kMiscRegs>();
    if (warp == kScaleWarp) {
      role_scales<kN>(p, tab, c);
      (void)meet();
    } else {
      const bool ok = meet();
      if (warp == kQueryWarp) {
        role_queries<kN>(p, tab, c);
      } else if (lane == 0 && ok) {
        if (c.rank == 0) {
          if (warp == kIssueWarp) role_issue<kN>(p, tab, c);
        } else {
          if (warp == kIssueWarp) role_forward_tiles(c, B_KL, B_KF);
          else role_forward_tiles(c, B_VL, B_VF);
          // this CTA's TMEM and shared memory are in use until the pair's last product is done
          if (warp == kIssueWarp) (void)mbar_wait_drain(c.bar(B_DRAIN), 0, kShDrainNs);
        }
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kN == 2) cluster_sync_all();  // no arrival from the other CTA is still on its way
  tc_fence_after();
  if (warp == kIssueWarp) {
    if constexpr (kN == 2) tmem_dealloc_pair(c.tm, 512);
    else tmem_dealloc(c.tm, 512);
  }
}
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPreThreads, 1)
    prefix_pair_kernel(const __grid_constant__ SharedParams p, const __grid_constant__ SharedSeqs tab) {
  prefix_pass<2>(p, tab);
}
__global__ void __launch_bounds__(kPreThreads, 1)
    prefix_one_kernel(const __grid_constant__ SharedParams p, const __grid_constant__ SharedSeqs tab) {
  prefix_pass<1>(p, tab);
}

// ====================================================================
// Each sequence's own keys
// ====================================================================
// CTA = (sequence, kv head, chunk of its visible blocks); its four warps take
// the blocks in turn.  Products as in the decode kernel, on mma.sync in the
// transposed orientation, S^T = K Q^T and O^T = V^T P^T: keys and dims fill M,
// the G <= 8 query rows N.  A warp's blocks come by TMA into two stages of its
// own, K and V with a barrier each, a stage's K filled again as soon as its
// scores are done: one to two blocks a warp are always on their way.  Which dims
// a thread's operands hold is free as long as Q and O agree: chosen so that its
// 16-byte reads of the 128-byte swizzled rows have no bank conflicts.
// Bound by memory where there is enough of it: 100 sequences of 1500 keys, 8 kv
// heads (626 MB) in 115 us, 5.4 TB/s; short passes by the latency of a CTA's start
// (~4.5 us) and of a block in a warp (~2 us: load, products, softmax, products).
// Straight from global memory into registers, half a block ahead, spilled at 168
// registers and took 41 us for 48 windowed sequences, with TMA 38.8.
constexpr int kOwnWarps = 4;
constexpr int kOwnStage = 8192;                              // K and V of a block, each two halves of [16][128]
constexpr int kOwnRing = 2 * kOwnStage;                      // a warp's; at the end its partial output [8][kOwnPitch]
constexpr int kOwnPitch = kHeadDim + 4;
constexpr int kOwnQ = kOwnWarps * kOwnRing;                  // [16][32] uint2: Q's fragments
constexpr int kOwnRow = kOwnQ + 16 * 32 * 8;                 // [8] the rows' factors
constexpr int kOwnML = kOwnRow + 8 * 4;                      // [2][warps][8] the warps' references and sums
constexpr int kOwnBar = kOwnML + 2 * kOwnWarps * 8 * 4;      // [warps][stage][K, V]
constexpr int kOwnSmem = kOwnBar + kOwnWarps * 4 * 8;
static_assert(kOwnSmem * kShOwnPerSm <= 224 * 1024 && 8 * kOwnPitch * 4 <= kOwnRing && kOwnBar % 8 == 0, "shared memory");

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Dims 4 dq .. + 3 of a row's output: its unnormalised sum over the softmax's.
__device__ __forceinline__ void store_row(const SharedParams& p, int row, int g, int r, int dq, const float4 acc, float l) {
  const float il = l > 0.f ? 1.f / l : 0.f;
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * il, acc.y * il), b = __floats2bfloat162_rn(acc.z * il, acc.w * il);
  *reinterpret_cast<uint2*>(p.out + ((size_t)row * p.HQ + (size_t)g * p.G + r) * kHeadDim + 4 * dq) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__global__ void __launch_bounds__(kOwnWarps * 32, kShOwnPerSm) own_kernel(const __grid_constant__ SharedParams p,
                                                             const __grid_constant__ SharedSeqs tab,
                                                             const __grid_constant__ DecodeMaps maps) {
  extern __shared__ __align__(1024) uint8_t raw[];
  dependents_may_start();
  const uint32_t sb = smem_u32(raw);
  if (sb & 1023u) {  // every thread: nothing was started
    if (threadIdx.x == 0) atomicCAS(p.err, 0, DEV_ERR_LAYOUT);
    return;
  }
  uint2* qf = reinterpret_cast<uint2*>(raw + kOwnQ);
  float* rowc = reinterpret_cast<float*>(raw + kOwnRow);
  float (*wm)[8] = reinterpret_cast<float(*)[8]>(raw + kOwnML);
  float (*wl)[8] = wm + kOwnWarps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  // the CTA's sequence (listed for the launch's first CTAs), kv head and chunk
  int lo = 0, hi = p.n_seq - 1;
  if ((int)blockIdx.x < kShOwnListed) lo = hi = tab.own_seq[blockIdx.x];
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.HKV * tab.s[mid].z <= (int)blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const int4 sq = tab.s[lo];
  const int t = sq.y - 1;
  const ShOwn own = shared_own(sq.y, sq.w, p.first_blk, p.S, p.W);
  const int at = (int)blockIdx.x - p.HKV * sq.z;
  const int ch = at / p.HKV, g = at - ch * p.HKV;  // the heads of a chunk side by side: they read the same DRAM pages
  const int b0 = ch * p.chunk, b1 = min(own.n, b0 + p.chunk);
  // this warp's pages, one per lane (at most 32 blocks a warp)
  auto block_of = [&](int b) { return b < own.sink ? p.first_blk + b : own.lo + (b - own.sink); };
  const int mine = b0 + warp + kOwnWarps * lane;
  int page = -1;
  if (mine < b1) {
    const int lb = block_of(mine);
    page = __ldg(p.block_table + (lb < p.prefix_blk ? 0 : (size_t)(p.bt_row0 + lo) * p.bt_stride) + lb);
    if (page < 0 || page >= p.n_pool) {
      page = -1;
      record_bad_page(p.err);
    }
  }
  const int n_it = b1 > b0 + warp ? (b1 - b0 - warp + kOwnWarps - 1) / kOwnWarps : 0;
  const uint32_t ring = sb + warp * kOwnRing, bars = sb + kOwnBar + 32 * warp;
  // a block of a bad page (skipped below) loads page 0
  auto page_of = [&](int it) { return max(0, __shfl_sync(kAllLanes, page, it)); };
  auto load = [&](int it, int v) {  // K or V of block it into its stage
    const int phys = page_of(it);
    if (lane == 0) {
      const uint32_t dst = ring + (it & 1) * kOwnStage + v * (kOwnStage / 2), bar = bars + 16 * (it & 1) + 8 * v;
      const CUtensorMap* map = v ? &maps.v : &maps.k;
      mbar_expect_tx(bar, kOwnStage / 2);
      tma_load_3d(dst, map, bar, 0, g, phys * kPage);
      tma_load_3d(dst + kOwnStage / 4, map, bar, 128, g, phys * kPage);
    }
  };
  if (lane == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  for (int it = 0; it < 2 && it < n_it; ++it) {
    load(it, 0);
    load(it, 1);
  }
  {  // the G query rows as B fragments: thread row r, dims [16 c, 16 c + 16)
    const int r = threadIdx.x >> 4, cc = threadIdx.x & 15;
    float v[16];
    float am = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.f;
    if (r < p.G) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + ((size_t)sq.x * p.HQ + (size_t)g * p.G + r) * kHeadDim + 16 * cc);
      float a[8], b[8];
      unpack8(__ldg(src), a);
      unpack8(__ldg(src + 1), b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = a[e], v[8 + e] = b[e], am = fmaxf(am, fmaxf(fabsf(a[e]), fabsf(b[e])));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(kAllLanes, am, o));
    const int k = row_shift(am);
    const float mul = pow2i(k);
#pragma unroll
    for (int m = 0; m < 4; ++m)
      qf[(4 * (2 * (cc >> 3) + (cc & 1)) + m) * 32 + 4 * r + (cc >> 1 & 3)] =
          make_uint2(pack_f16x2(v[4 * m] * mul, v[4 * m + 1] * mul), pack_f16x2(v[4 * m + 2] * mul, v[4 * m + 3] * mul));
    if (cc == 0) rowc[r] = r < p.G ? pow2i(-k) * p.sm_scale_log2 : 0.f;
  }
  __syncthreads();
  const float c_lo = rowc[2 * tq], c_hi = rowc[2 * tq + 1];
  float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;
  int ev = -100;
  float o[16][4];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  // the scales of keys gq and gq + 8, a block ahead
  float ks0 = 0.f, ks1 = 0.f, vr0 = 0.f, vr1 = 0.f;
  auto load_scales = [&](int it) {
    const size_t s0 = ((size_t)page_of(it) * kPage + gq) * p.HKV + g;
    ks0 = __ldg(p.k_scale + s0);
    ks1 = __ldg(p.k_scale + s0 + 8 * (size_t)p.HKV);
    vr0 = __ldg(p.v_scale + s0);
    vr1 = __ldg(p.v_scale + s0 + 8 * (size_t)p.HKV);
  };
  if (n_it > 0) load_scales(0);
  const WaitCtl wc{p.err, p.wait_ns};
  int it = 0, n_k = min(n_it, 2), n_v = n_k;  // copies issued
  for (; it < n_it; ++it) {
    const int b = b0 + warp + kOwnWarps * it;
    const uint32_t stage = ring + (it & 1) * kOwnStage, bar = bars + 16 * (it & 1);
    const bool good = __shfl_sync(kAllLanes, page, it) >= 0;
    float sacc[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m) sacc[m][0] = sacc[m][1] = sacc[m][2] = sacc[m][3] = 0.f;
    const float s_k0 = ks0, s_k1 = ks1, s_v0 = vr0, s_v1 = vr1;
    if (it + 1 < n_it) load_scales(it + 1);
    if (!__all_sync(kAllLanes, mbar_wait(bar, (it >> 1) & 1, wc, 120))) break;
    // K: rows gq and gq + 8, dims 128 (j / 2) + 32 tq + 16 (j % 2)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t at = stage + (j >> 1) * 2048 + gq * 128 + (((2 * tq + (j & 1)) ^ gq) << 4);
      const uint4 u0 = lds_u32x4(at), u1 = lds_u32x4(at + 1024);
      const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w};
      const uint32_t w1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint32_t x0 = w0[m] ^ 0x80808080u, x1 = w1[m] ^ 0x80808080u;
        const uint32_t a[4] = {lo_pair(x0), lo_pair(x1), hi_pair(x0), hi_pair(x1)};
        const uint2 bq = qf[(4 * j + m) * 32 + lane];
        mma16816(sacc[m], a, bq.x, bq.y);
      }
    }
    __syncwarp();
    if (n_k < n_it) load(n_k++, 0);
    float sc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[e] = (sacc[0][e] + sacc[1][e]) + (sacc[2][e] + sacc[3][e]);
    const int lb = block_of(b);
    const bool v0 = good && lb * kPage + gq <= t, v1 = good && lb * kPage + gq + 8 <= t;
    const float y0 = v0 ? sc[0] * s_k0 * c_lo : -INFINITY, y1 = v0 ? sc[1] * s_k0 * c_hi : -INFINITY;
    const float y2 = v1 ? sc[2] * s_k1 * c_lo : -INFINITY, y3 = v1 ? sc[3] * s_k1 * c_hi : -INFINITY;
    float bm_lo = fmaxf(y0, y2), bm_hi = fmaxf(y1, y3);
    float bv = fmaxf(v0 ? s_v0 : 0.f, v1 ? s_v1 : 0.f);
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
      bm_lo = fmaxf(bm_lo, __shfl_xor_sync(kAllLanes, bm_lo, sh));
      bm_hi = fmaxf(bm_hi, __shfl_xor_sync(kAllLanes, bm_hi, sh));
      bv = fmaxf(bv, __shfl_xor_sync(kAllLanes, bv, sh));
    }
    const float mn_lo = fmaxf(m_lo, bm_lo), mn_hi = fmaxf(m_hi, bm_hi);  // -inf only while every page was bad
    const float ml = mn_lo == -INFINITY ? 0.f : mn_lo, mh = mn_hi == -INFINITY ? 0.f : mn_hi;
    const int ev_n = max(ev, exp_above(bv));
    const float vfix = ev_n > ev ? (ev_n - ev > 126 ? 0.f : pow2i(ev - ev_n)) : 1.f;
    ev = ev_n;
    const float vnorm = pow2i(-ev);
    const float al_lo = ex2f(m_lo - ml), al_hi = ex2f(m_hi - mh);
    m_lo = mn_lo;
    m_hi = mn_hi;
    const float p0 = ex2f(y0 - ml), p1 = ex2f(y1 - mh), p2 = ex2f(y2 - ml), p3 = ex2f(y3 - mh);
    l_lo = l_lo * al_lo + (p0 + p2);
    l_hi = l_hi * al_hi + (p1 + p3);
    if (__any_sync(kAllLanes, al_lo != 1.f || al_hi != 1.f || vfix != 1.f)) {
      const float f_lo = al_lo * vfix, f_hi = al_hi * vfix;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        o[i][0] *= f_lo;
        o[i][1] *= f_hi;
        o[i][2] *= f_lo;
        o[i][3] *= f_hi;
      }
    }
    const float vs0 = v0 ? s_v0 * vnorm : 0.f, vs1 = v1 ? s_v1 * vnorm : 0.f;
    const uint32_t pb0 = transpose8x8(pack_f16x2(v0 ? p0 * vs0 : 0.f, v0 ? p1 * vs0 : 0.f));
    const uint32_t pb1 = transpose8x8(pack_f16x2(v1 ? p2 * vs1 : 0.f, v1 ? p3 * vs1 : 0.f));
    if (!__all_sync(kAllLanes, mbar_wait(bar + 8, (it >> 1) & 1, wc, 121))) break;
    // V: keys 2tq, + 1, + 8, + 9, dims 128 h + 16 gq + 2 (mt % 8) (row gq of m-tile mt = 8 h ..) and + 1 (row gq + 8)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 2 * tq + (k & 1);
        const uint4 u = lds_u32x4(stage + 4096 + h * 2048 + (k >> 1) * 1024 + r * 128 + ((gq ^ r) << 4));
        w[k][0] = u.x, w[k][1] = u.y, w[k][2] = u.z, w[k][3] = u.w;
      }
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const int i = 4 * h + ii;
        const uint32_t lo01 = __byte_perm(w[0][ii], w[1][ii], 0x5140) ^ 0x80808080u;
        const uint32_t hi01 = __byte_perm(w[0][ii], w[1][ii], 0x7362) ^ 0x80808080u;
        const uint32_t lo89 = __byte_perm(w[2][ii], w[3][ii], 0x5140) ^ 0x80808080u;
        const uint32_t hi89 = __byte_perm(w[2][ii], w[3][ii], 0x7362) ^ 0x80808080u;
        const uint32_t a0[4] = {lo_pair(lo01), hi_pair(lo01), lo_pair(lo89), hi_pair(lo89)};
        mma16816(o[2 * i], a0, pb0, pb1);
        const uint32_t a1[4] = {lo_pair(hi01), hi_pair(hi01), lo_pair(hi89), hi_pair(hi89)};
        mma16816(o[2 * i + 1], a1, pb0, pb1);
      }
    }
    __syncwarp();
    if (n_v < n_it) load(n_v++, 1);
  }
  if (it < n_it) {  // a wait gave up: no copy may be in flight when the CTA leaves
    for (int v = 0; v < 2; ++v)
      for (int n = v ? n_v : n_k, i = max(0, n - 2); i < n; ++i)  // the last of each stage
        (void)mbar_wait_drain(bars + 16 * (i & 1) + 8 * v, (i >> 1) & 1, kShDrainNs);
    __syncwarp();
  }
#pragma unroll
  for (int sh = 4; sh < 32; sh <<= 1) {
    l_lo += __shfl_xor_sync(kAllLanes, l_lo, sh);
    l_hi += __shfl_xor_sync(kAllLanes, l_hi, sh);
  }
  if (gq == 0) {
    wm[warp][2 * tq] = m_lo;
    wm[warp][2 * tq + 1] = m_hi;
    wl[warp][2 * tq] = l_lo;
    wl[warp][2 * tq + 1] = l_hi;
  }
  const float up = pow2i(max(ev, -126));
  float* part = reinterpret_cast<float*>(raw + warp * kOwnRing);  // over the stages: all copies have landed and are read
  __syncwarp();
#pragma unroll
  for (int mt = 0; mt < 16; ++mt) {  // rows 2tq, 2tq+1
    const int d = 128 * (mt >> 3) + 16 * gq + 2 * (mt & 7);
    *reinterpret_cast<float2*>(part + 2 * tq * kOwnPitch + d) = make_float2(o[mt][0] * up, o[mt][2] * up);
    *reinterpret_cast<float2*>(part + (2 * tq + 1) * kOwnPitch + d) = make_float2(o[mt][1] * up, o[mt][3] * up);
  }
  __syncthreads();
  // the warps' parts, in a fixed order; thread (row i % 8, dims 4 (i / 8 + 16 n))
  const int r = threadIdx.x & 7;
  float mx = -INFINITY, ls = 0.f, f[kOwnWarps];
#pragma unroll
  for (int w = 0; w < kOwnWarps; ++w) mx = fmaxf(mx, wm[w][r]);
#pragma unroll
  for (int w = 0; w < kOwnWarps; ++w) {
    f[w] = wm[w][r] == -INFINITY ? 0.f : ex2f(wm[w][r] - mx);
    ls += f[w] * wl[w][r];
  }
  float4 part_o[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int dq = (threadIdx.x >> 3) + 16 * n;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(raw + w * kOwnRing + 4 * (r * kOwnPitch + 4 * dq));
      acc.x = fmaf(f[w], v.x, acc.x);
      acc.y = fmaf(f[w], v.y, acc.y);
      acc.z = fmaf(f[w], v.z, acc.z);
      acc.w = fmaf(f[w], v.w, acc.w);
    }
    part_o[n] = acc;
  }
  if (p.merge_ways == 0) {  // no prefix pass, and a row's keys are one chunk: its output
    if (r < p.G) {
#pragma unroll
      for (int n = 0; n < 4; ++n) store_row(p, sq.x, g, r, (threadIdx.x >> 3) + 16 * n, part_o[n], ls);
    }
    return;
  }
#pragma unroll
  for (int n = 0; n < 4; ++n) p.own_o[((size_t)blockIdx.x * 64 + (threadIdx.x >> 3) + 16 * n) * 8 + r] = part_o[n];
  if (threadIdx.x < 8) p.own_ml[(size_t)blockIdx.x * 8 + r] = make_float2(mx, ls);
  // This grid's end has to mean that the prefix pass has ended too.  One CTA
  // waits for it, the last: the others leave their places to those still to come.
  if (blockIdx.x == gridDim.x - 1) wait_for_previous();
}

// ====================================================================
// Merge
// ====================================================================
// CTA = (sequence, kv head, 32 of the dims); thread (row i % G, dims 4 (i / G %
// 8), every merge_ways-th partial from i / (8 G) on), then the ways' parts
// through shared memory in a fixed order.  Bound by the latency of the partials'
// loads: the ways (as many as give a thread about four partials) and four loads
// a thread keep them in flight together.  (64 dims and 8 ways at most: 53 us
// instead of 51 for 64 sequences on 32768 keys, 37.5 instead of 35.3 for 9 on
// 131072, whose rows have 150 partials.)
constexpr int kMergeMostWays = 16;
constexpr int kMergeDims = 32;

__global__ void __launch_bounds__(8 * kMergeDims / 4 * kMergeMostWays) merge_kernel(const __grid_constant__ SharedParams p,
                                                                    const __grid_constant__ SharedSeqs tab) {
  __shared__ float4 acc_sh[kMergeMostWays - 1][kMergeDims / 4 * 8];
  __shared__ float2 ml_sh[kMergeMostWays - 1][kMergeDims / 4 * 8];
  const int s = blockIdx.x / p.HKV, g = blockIdx.x % p.HKV;
  const int slot = threadIdx.x % (kMergeDims / 4 * p.G), way = threadIdx.x / (kMergeDims / 4 * p.G);
  const int r = slot & (p.G - 1), dq = blockIdx.y * (kMergeDims / 4) + (slot >> p.log2_g);
  const int4 sq = tab.s[s];
  const ShOwn own = shared_own(sq.y, sq.w, p.first_blk, p.S, p.W);
  const int n_own = (own.n + p.chunk - 1) / p.chunk, own0 = p.HKV * sq.z + g;
  int n_pre = 0, pre0 = 0, prow = 0, rows = 0;
  if (p.n_grp > 0) {
    const int unit = p.n_cta * kRows, rg = (s * p.G) / unit;
    const ShGroup grp = tab.grp[rg];
    if (grp.n_blk > 0) {
      const int c0 = tab.first_unit[g * p.n_grp + rg], c1 = tab.last_unit[g * p.n_grp + rg];
      n_pre = c1 - c0 + 1;
      pre0 = c0 + g * p.n_grp + rg;
      prow = s * p.G - rg * unit + r;
      rows = unit;
    }
  }
  // partial i of the row: the prefix's, then its own keys'
  const int n = n_pre + n_own;
  const float2* pm = p.pre_ml + (size_t)pre0 * rows + prow;
  const float4* po = p.pre_o + ((size_t)pre0 * 64 + dq) * rows + prow;
  const float2* om = p.own_ml + (size_t)own0 * 8 + r;
  const float4* oo = p.own_o + ((size_t)own0 * 64 + dq) * 8 + r;
  wait_for_previous();
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float2 ml, const float4 v) {
    if (ml.x == -INFINITY) return;  // no visible key
    const float mn = fmaxf(m, ml.x);
    const float f = m == -INFINITY ? 0.f : ex2f(m - mn), w = ex2f(ml.x - mn);
    m = mn;
    l = fmaf(w, ml.y, l * f);
    acc.x = fmaf(w, v.x, acc.x * f);
    acc.y = fmaf(w, v.y, acc.y * f);
    acc.z = fmaf(w, v.z, acc.z * f);
    acc.w = fmaf(w, v.w, acc.w * f);
  };
  for (int i0 = way; i0 < n; i0 += 4 * p.merge_ways) {
    float2 ml[4];
    float4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e * p.merge_ways;
      ml[e] = make_float2(-INFINITY, 0.f);
      v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n_pre) {
        ml[e] = __ldcg(pm + (size_t)i * rows);
        v[e] = __ldcg(po + (size_t)i * 64 * rows);
      } else if (i < n) {
        ml[e] = __ldcg(om + (size_t)(i - n_pre) * p.HKV * 8);
        v[e] = __ldcg(oo + (size_t)(i - n_pre) * p.HKV * 64 * 8);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) add(ml[e], v[e]);
  }
  if (way > 0) {
    acc_sh[way - 1][slot] = acc;
    ml_sh[way - 1][slot] = make_float2(m, l);
  }
  __syncthreads();
  if (way > 0) return;
  for (int w = 0; w < p.merge_ways - 1; ++w) add(ml_sh[w][slot], acc_sh[w][slot]);
  store_row(p, sq.x, g, r, dq, acc, l);
}

template <typename... Params>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t st, const Params&... params) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, params...);
}

}  // namespace

cudaError_t launch_decode_shared(const SharedParams& p, const SharedSeqs& t, const DecodeMaps& maps, cudaStream_t st) {
  cudaError_t e;
  const int own_grid = p.HKV * p.chunks_head;
  if ((e = cudaFuncSetAttribute(own_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOwnSmem)) != cudaSuccess) return e;
  if (p.n_grp > 0 && p.tiles_head > 0) {
    auto* kernel = p.n_cta == 2 ? prefix_pair_kernel : prefix_one_kernel;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPreSmem)) != cudaSuccess) return e;
    kernel<<<p.n_cta * p.n_units, kPreThreads, kPreSmem, st>>>(p, t);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_after(own_kernel, dim3((unsigned)own_grid), kOwnWarps * 32, kOwnSmem, st, p, t, maps)) != cudaSuccess)
      return e;
  } else {
    own_kernel<<<own_grid, kOwnWarps * 32, kOwnSmem, st>>>(p, t, maps);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (p.merge_ways == 0) return cudaSuccess;
  return launch_after(merge_kernel, dim3((unsigned)(p.n_seq * p.HKV), kHeadDim / kMergeDims),
                      kMergeDims / 4 * p.G * p.merge_ways, 0, st,
                      p, t);
}

}  // namespace pa
