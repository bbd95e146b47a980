// Declarations shared by the C-ABI host code and the shared-prefix decode
// kernels (pa_shared.cu).  Not part of the public interface.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pa_internal.h"
#include "pa_tiles.cuh"

namespace pa {

constexpr int kShSeqs = 512;                        // sequences per launch, their table in its parameters
constexpr int kShGroups = kShSeqs * 8 / (2 * kRows);  // row groups of one kv head at most (8 q heads a kv head)

// Blocks of the prefix that some row of a group of query rows (128 for each CTA
// that works on it) sees: the sink run [0, sink) and the run [lo, prefix blocks).
struct ShGroup {
  int x0;    // tiles of the head's earlier groups
  int sink;
  int lo;
  int n_blk; // sink + prefix blocks - lo
};

constexpr int kShUnits = 256;  // units (a CTA or a pair of them) of the prefix pass at most

constexpr int kShOwnListed = 1024;
constexpr int kShOwnPerSm = 3;  // CTAs of the per-sequence pass on an SM at a time

struct SharedSeqs {
  // {row in q / out, context length, chunks of the earlier sequences (per kv head), first block of its window}
  int4 s[kShSeqs];
  ShGroup grp[kShGroups];
  // The prefix pass's tiles (fewer than 2^30), head-major and group-major, laid
  // end to end: unit c computes tiles [cut[c], cut[c + 1]); group j (head-major)
  // lies in units first_unit[j] .. last_unit[j].
  int cut[kShUnits + 1];
  uint8_t first_unit[8 * kShGroups], last_unit[8 * kShGroups];
  uint16_t own_seq[kShOwnListed];  // sequence of the per-sequence pass's first CTAs (a search finds the others')
};

struct SharedParams {
  const __nv_bfloat16* q;  // [rows][HQ][256]
  __nv_bfloat16* out;
  const int8_t* k_pool;    // [n_pool][16][HKV][256]
  const int8_t* v_pool;
  const float* k_scale;    // [n_pool][16][HKV]
  const float* v_scale;
  const int32_t* block_table;
  int bt_stride, n_pool, bt_row0;
  int n_seq, HQ, HKV, G, S, W;
  int log2_g;              // G = q heads per kv head is 1, 2, 4 or 8
  int prefix_blk;          // blocks of the shared prefix; their pages are block_table row 0's
  int first_blk;           // the per-sequence pass starts at this block: prefix_blk, or 0 without a prefix pass
  int n_grp;               // row groups per kv head (0: no prefix pass)
  int n_cta;               // CTAs of a unit of the prefix pass, 1 or 2: groups of 128 n_cta rows
  int tiles_head;          // 128-key tiles of all groups of one kv head
  int n_units;             // units of the prefix pass
  int chunk;               // blocks per CTA of the per-sequence pass
  int chunks_head;         // its CTAs per kv head
  int merge_ways;          // threads that share a row's partials in the merge, 1 to 16; 0: no merge, every row is one CTA's
  float sm_scale_log2;
  // Partials: per row the reference (log2 units) and sum of its softmax, and
  // its unnormalised output, 4 dims x rows side by side.  Prefix: the partial
  // of unit c for group j (head-major) is number c + j; own keys: the CTA's number.
  float4* pre_o;           // [c + j][64][128 n_cta]
  float2* pre_ml;          // [c + j][128 n_cta]
  float4* own_o;           // [cta][64][8]
  float2* own_ml;          // [cta][8]
  int* err;
  unsigned long long wait_ns;
};

// Blocks of a sequence that the per-sequence pass visits, from block `first` on.
struct ShOwn {
  int sink, lo, n;  // sink blocks first .. first + sink, then blocks from lo on; n in all
};
PA_HD ShOwn shared_own(int n_ctx, int win_lo, int first, int S, int W) {
  ShOwn o;
  o.sink = W > 0 ? imax(0, imin(S, win_lo) - first) : 0;
  o.lo = imax(win_lo, first);
  o.n = o.sink + (n_ctx - 1) / kPage + 1 - o.lo;
  return o;
}
PA_HD int shared_win_lo(int n_ctx, int W) { return W > 0 ? imax(0, (n_ctx - 1) / kPage + 1 - W) : 0; }

// maps: the pool as uint8 [n_pool * 16][HKV][256], boxes of 16 tokens, one head, 128 dims, 128-byte swizzle.
cudaError_t launch_decode_shared(const SharedParams& p, const SharedSeqs& t, const DecodeMaps& maps, cudaStream_t st);

}  // namespace pa
