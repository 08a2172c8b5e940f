// Internal interface of the many-row attention kernel (kvq_rows.cu) and the merge of its
// partials (kvq_rows_merge.cu).
#pragma once

#include <math.h>

#include "kvq_internal.h"

namespace kvq {

constexpr int kRowTile = 256;   // query rows of one unit (two TMEM row tiles of 128)
constexpr int kKvTile = 128;    // positions: one K / V block for each of two streams
constexpr int kTargetCtas = 148;  // SMs of a B200: one CTA each

// Attention of many query rows over groups of positions.  Group g owns the tokens
// offsets[g] .. offsets[g + 1] - 1 (a row is one query head of one token; the heads of one
// KV head are consecutive rows) and the positions 0 .. lens[g] - 1 of its pages.
struct RowsArgs {
  kvq_cache_desc desc;
  const void* q;           // fp16 [n_tokens][num_q_heads][head_dim]
  int n_tokens, num_q_heads, group;
  const void* k_codes;
  const void* k_scales;
  const void* v_codes;
  const void* v_scales;
  const int32_t* table;    // [num_groups][max_pages], or null: pages g*max_pages ..
  int max_pages;
  const int32_t* lens;     // [num_groups]
  int max_len;
  const int32_t* offsets;  // [num_groups + 1], or null: one group of every token
  int num_groups;
  int causal;              // token i of n sees the positions < lens - n + i + 1; else all
  float sm_scale;
  int splits;              // splits of a unit at the most
  int min_chunk;           // each unit's positions are cut at multiples of a chunk chosen on the
                           // device (of kKvTile, at least this): the shortest whose units all run at
                           // once on `ctas` CTAs.  One split: max_len.
  int ctas;
  int row_tiles;           // row tiles of all groups at the most
  int32_t* chunk_out;      // the chunk, for the merge
  // out != null: one split, the rows are normalized and written here; otherwise partials:
  float* part_o;           // [n_tokens][num_q_heads][splits][head_dim], unnormalized
  float* part_m;           // [n_tokens][num_q_heads][splits] running maximum, log2 units
  float* part_l;           // [n_tokens][num_q_heads][splits]
  void* out;
  int out_f16;
  uint32_t* flags;
};

// Decode of single tokens over their own positions in the same launch (kvq_own.cuh): token b's
// positions 0 .. seq_lens[b] - 1, cut at multiples of split.  units = 0: none has any; seq_lens
// null: not a prefix decode.
struct OwnArgs {
  int64_t units;           // n_tokens * num_kv_heads * max_splits, one warp each
  const int32_t* table;    // [n_tokens][max_pages], or null: pages b*max_pages ..
  int max_pages;
  const int32_t* seq_lens;
  int max_seq_len, split, max_splits;
  float* part_o;           // [n_tokens][num_q_heads][max_splits][head_dim], unnormalized
  float* part_m;           // [n_tokens][num_q_heads][max_splits] maximum, log2 units
  float* part_l;
};

// The split of a request: row tiles, splits and positions per split.
struct RowsPlan {
  int row_tiles, splits, min_chunk, ctas;
};
RowsPlan plan_rows(int num_kv_heads, int group, int n_tokens, int num_groups, int max_len, int ctas);
size_t rows_partial_bytes(int n_tokens, int num_q_heads, int head_dim, int splits);
// Positions per split of the own part, and the CTAs it takes.
int plan_own(int num_kv_heads, int batch, int max_seq_len, int* ctas);

int launch_rows(const RowsArgs& a, const OwnArgs& own, cudaStream_t stream);
// Merge of the partials of a rows launch (own.seq_lens: those of the own positions as well) into
// the normalized output; lut4 is rotated back.
int launch_rows_merge(const RowsArgs& a, const OwnArgs& own, void* out, int out_f16, cudaStream_t stream);

// The visible positions of token i of a group of n tokens and `len` positions.
__host__ __device__ inline int row_limit(int len, int n, int i, int causal) {
  if (!causal) return len;
  const int lim = len - n + i + 1;
  return lim < 0 ? 0 : lim;
}

// What a row of weights summing to l is multiplied by; empty: no maximum, so no position.  The
// largest weight of any other row is 2^7 or more: a sum below 1 means that the weights have left
// fp16 downwards (scores beyond 2^27, where fp32 has steps of 8 and more), a NaN that a score was
// one; neither may pass for a result.
__device__ __forceinline__ float row_scale(float l, bool empty) {
  return l >= 1.f ? 1.f / l : empty && l == 0.f ? 0.f : NAN;
}

}  // namespace kvq
