// Declarations shared by the C-ABI host code and the norm / rotation / append
// kernel (pa_qkv.cu).  Not part of the public interface.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/pa.h"

namespace pa {

// bf16 rows [token][head][256] at element strides.
struct RowsIn {
  const __nv_bfloat16* p;
  long long ts, hs;
};

struct QkvParams {
  RowsIn q, k, v;                    // p == nullptr: no such rows
  const __nv_bfloat16* qw;           // [256] gains, or nullptr (1)
  const __nv_bfloat16* kw;
  float w_off;                       // added to the gains
  float eps;
  pa_rope rope;                      // rot_dim 0: no rotation
  const int32_t* pos;                // [n_axes][pos_stride] by row, or nullptr: the token's own position
  long long pos_stride;
  __nv_bfloat16* q_out;              // [row][HQ][256]
  __nv_bfloat16* k_out;              // [row][HKV][256]; the append writes the pool instead
  int n_q, n_k, n_v;                 // rows per token of each kind
  int n_tok, parts, rows_per_part;   // a warp's item: one token, rows_per_part of its rows
  // append only
  int n_seq, same_len;               // same_len: every sequence's token count if they are all equal, else 0
  const int32_t* block_table;
  int bt_stride, bt_row0, n_pool, HKV;
  int8_t* k_pool;
  int8_t* v_pool;
  float* k_scale;
  float* v_scale;
  int* err;
};

// Sequences of one append launch, carried in its parameters: {first row, first
// position, tokens of the launch's earlier sequences, 0}.
constexpr int kQkvSeqs = 512;
// A smaller table for the common small batches, 256 bytes of parameters and not 8 KB: one call, waited for, of one to
// 16 sequences takes 27.6 us, with the large one 28.5; among others, and on the device, both take the same.
constexpr int kQkvFewSeqs = 16;
template <int N>
struct QkvSeqs {
  int4 s[N];
};

// Rows a warp handles one after another, for n_tok tokens of `rows` rows each.
int qkv_rows_per_part(long long n_tok, int rows, int n_sm);
cudaError_t launch_qk_norm_rope(const QkvParams& p, int n_sm, cudaStream_t st);
cudaError_t launch_qkv_append(const QkvParams& p, const QkvSeqs<kQkvSeqs>& seqs, int n_sm, cudaStream_t st);

}  // namespace pa
