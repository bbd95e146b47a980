// Declarations shared by the C-ABI host code and the kernels of the 4-bit pool
// (pa_kv4.cu, pa_kv4_decode.cu).  Not part of the public interface.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/pa.h"
#include "pa_internal.h"
#include "pa_qkv.h"

namespace pa {

// A tile: one kv head's 16 tokens of a page (include/pa.h has the format).
constexpr int kT4V = 2048;       // V codes, behind K's
constexpr int kT4Block = 4096;   // K block scales, V's 256 bytes on
constexpr int kT4Row = 4608;     // K row scales, V's 64 bytes on
constexpr int kT4Bytes = PA_KV4_TILE_BYTES;
static_assert(kT4Bytes == 4736 && kT4Bytes % 128 == 0, "tiles of whole 128-byte lines");

// New tokens of a batch of sequences into the pool (append), or out of it (gather).
struct Kv4RowsParams {
  RowsIn k, v;                // append: the rows
  __nv_bfloat16* k_out;       // gather: [row][HKV][256], or nullptr
  __nv_bfloat16* v_out;
  uint8_t* pool;              // [n_pool][HKV][kT4Bytes]; the gather only reads it
  const int32_t* block_table;
  int bt_stride, bt_row0, n_pool, HKV;
  int n_seq, n_tok, same_len; // of this launch; same_len: every sequence's token count if they are all equal, else 0
  int* err;
};
cudaError_t launch_kv4_append(const Kv4RowsParams& p, const QkvSeqs<kQkvSeqs>& seqs, cudaStream_t st);
cudaError_t launch_kv4_gather(const Kv4RowsParams& p, const QkvSeqs<kQkvSeqs>& seqs, cudaStream_t st);

// The widening pass of the prefill (WidenParams) from the 4-bit pool; its int8 pools and scales are not read.
cudaError_t launch_widen_kv4(const WidenParams& p, const uint8_t* pool, cudaStream_t st);

// Decode: the visible blocks of a (sequence, kv head) pair are cut into runs, a warp each.
constexpr int kKv4Seqs = 512;      // sequences per launch, their table carried in the launch's parameters
constexpr int kKv4Ctas = 1536;     // CTAs of a launch, likewise
constexpr int kKv4Part = 16 * 32;  // float4 of a partial: 8 rows x 256
template <int kSeqs, int kCtas>
struct Kv4DecodeTable {
  static constexpr bool kHints = kCtas > 1;
  int4 seq[kSeqs];          // {row of the token in q / out, context length, runs of the earlier sequences, runs of a pair}
  uint16_t cta_seq[kCtas];  // sequence of CTA c's first run
};
using Kv4DecodeSeqs = Kv4DecodeTable<kKv4Seqs, kKv4Ctas>;
// A few sequences: a warp looks for its own from the first on, and the host copies 0.3 KB of parameters, not 11, twice.
constexpr int kKv4FewSeqs = 16;
struct Kv4DecodeParams {
  const __nv_bfloat16* q;  // [rows][HQ][256]
  __nv_bfloat16* out;      // [rows][HQ][256], may be q
  const uint8_t* pool;
  const int32_t* block_table;
  int bt_stride, n_pool;
  int n_seq, bt_row0;      // sequences of this launch, and the first one's block-table row
  int S, W;
  int HQ, HKV, G;
  int n_runs, most_runs;   // runs of the launch; of a pair, at most
  float sm_scale_log2;
  float* part;             // [n_runs][kKv4Part] float4
  float2* nw;              // [n_runs][8]: of each row the reference of its O, the logarithm of its sum of weights
  int* err;
  unsigned long long wait_ns;
};
cudaError_t launch_kv4_decode(const Kv4DecodeParams& p, const Kv4DecodeSeqs& seqs, cudaStream_t st);
int kv4_decode_warps(int n_sm);  // that the GPU holds at once
int kv4_decode_cta_warps();

}  // namespace pa
