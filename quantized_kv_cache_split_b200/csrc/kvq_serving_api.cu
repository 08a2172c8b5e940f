// C-ABI entry points of the serving operators: the page plan of a step, prompt attention and
// shared-prefix decode.  Argument validation, then the launches; nothing is launched on an error.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_plan.h"
#include "kvq_rows.h"

namespace kvq {
namespace {

constexpr int kMaxLen = 1 << 29;
constexpr int kChunkWord = 40;  // 32-bit word of the workspace header that holds the rows launch's chunk

// What kvq_prompt_attn and kvq_prefix_attn ask of a request besides its pointers.
int check_rows(const kvq_cache_desc* desc, int64_t n_tokens, int num_q_heads, int groups, int max_len) {
  const int st = check_desc(desc);
  if (st != KVQ_OK) return st;
  if (n_tokens < 0 || num_q_heads < 1 || groups < 0 || max_len < 0) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads % desc->num_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads / desc->num_kv_heads > KVQ_MAX_GROUP || groups > KVQ_MAX_BATCH || max_len > kMaxLen)
    return KVQ_ERR_UNSUPPORTED;
  if (n_tokens * num_q_heads > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

// lut4 rows are rotated back by the merge kernel, so they always go through it.
bool needs_merge(const kvq_cache_desc* desc, const RowsPlan& p) {
  return p.splits > 1 || desc->fmt == KVQ_FMT_LUT4;
}

// How prompt attention is cut.  Up to 512 positions in one piece, written to the output directly:
// the merge costs more than the split saves (200 tokens of 32 heads at 512 positions: 20.3 us against
// 24.9; from 1 to 8 requests of 1 to 200 tokens at 300 to 512 positions 2 to 7 us less or the same;
// at 1024 positions the split wins, 22.8 against 25.6 for 64 tokens).  lut4 output goes through the
// merge in any case and keeps its splits.
RowsPlan plan_prompt(const kvq_cache_desc* desc, int n_tokens, int num_q_heads, int batch, int max_seq_len) {
  RowsPlan p = plan_rows(desc->num_kv_heads, num_q_heads / desc->num_kv_heads, n_tokens, batch, max_seq_len, kTargetCtas);
  if (max_seq_len <= 4 * kKvTile && desc->fmt != KVQ_FMT_LUT4) {
    p.splits = 1;
    p.min_chunk = 4 * kKvTile;
  }
  return p;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// The two parts of prefix decode: how each is cut.  Blocks of either fill an SM, so the prefix gets
// the share of the SMs that its work is of all of it, and the own part's blocks run beside it on
// the others.  Work in microseconds of an SM as measured: a tile of 128 positions 2.1 and a block
// 10 for the prefix, a 64-position block of twelve own units 4 (8 for lut4).
struct PrefixPlan {
  RowsPlan rows;
  int own_split, own_splits;
};
PrefixPlan plan_prefix(const kvq_cache_desc* desc, int batch, int num_q_heads, int num_groups, int max_prefix_len,
                       int max_seq_len) {
  PrefixPlan p;
  int ctas = 0;
  p.own_split = plan_own(desc->num_kv_heads, batch, max_seq_len, &ctas);
  p.own_splits = (max_seq_len + p.own_split - 1) / p.own_split;
  const int group = num_q_heads / desc->num_kv_heads;
  const RowsPlan whole = plan_rows(desc->num_kv_heads, group, batch, num_groups, max_prefix_len, kTargetCtas);
  const double units = (double)whole.row_tiles * desc->num_kv_heads;
  const double prefix = units * ((max_prefix_len + kKvTile - 1) / kKvTile) * 2.1 + 10.0 * kTargetCtas;
  const double own = (double)ctas * (p.own_split / kTile) * (desc->fmt == KVQ_FMT_LUT4 ? 8.0 : 4.0);
  const int share = (int)(kTargetCtas * prefix / (prefix + own) + 0.5);
  p.rows = plan_rows(desc->num_kv_heads, group, batch, num_groups, max_prefix_len, std::max(share, kTargetCtas / 3));
  return p;
}

// Pointers into a rows workspace at `at`.
void set_partials(RowsArgs* r, uint8_t* at) {
  const size_t n = (size_t)r->n_tokens * r->num_q_heads * r->splits;
  r->part_o = reinterpret_cast<float*>(at);
  r->part_m = r->part_o + n * r->desc.head_dim;
  r->part_l = r->part_m + n;
}

// The lengths and offsets that no unit of a prefix decode looks at, because a bound of 0 leaves the
// prefixes (no row tiles) or the requests' own positions (no own units) without one.
__global__ void __launch_bounds__(256) check_kernel(const RowsArgs r, const OwnArgs own) {
  auto bad_len = [&](int len, int most, int pages) {
    return len < 0 || len > most || len > (int64_t)pages * r.desc.page_size;
  };
  bool bad = false;
  if (r.row_tiles == 0)
    for (int g = threadIdx.x; g < r.num_groups; g += 256) {
      const int first = r.offsets ? r.offsets[g] : 0, end = r.offsets ? r.offsets[g + 1] : r.n_tokens;
      bad |= first < 0 || end < first || end > r.n_tokens || bad_len(r.lens[g], r.max_len, r.max_pages);
    }
  if (own.units == 0)
    for (int b = threadIdx.x; b < r.n_tokens; b += 256) bad |= bad_len(own.seq_lens[b], own.max_seq_len, own.max_pages);
  if (bad) set_flag(r.flags, KVQ_FLAG_BAD_SEQLEN);
}

// The calls of the same names; flags: the device flag word, null for the workspace's.
int prompt_attn(const kvq_cache_desc* desc, const void* q, int32_t n_tokens,
                int32_t num_q_heads, const void* k_codes, const void* k_scales,
                const void* v_codes, const void* v_scales, const int32_t* page_table,
                int32_t max_pages, const int32_t* seq_lens, int32_t max_seq_len,
                const int32_t* token_offsets, int32_t batch, int32_t causal, float sm_scale,
                void* workspace, size_t workspace_bytes, void* out, int32_t out_type,
                uint32_t* flags, void* stream) {
  int st = check_rows(desc, n_tokens, num_q_heads, batch, max_seq_len);
  if (st != KVQ_OK) return st;
  if (max_pages < 1 || (causal != 0 && causal != 1) || (out_type != KVQ_OUT_F32 && out_type != KVQ_OUT_F16) ||
      !isfinite(sm_scale))
    return KVQ_ERR_INVALID_ARG;
  if (batch == 0 || n_tokens == 0) return KVQ_OK;  // (buffers of no elements may be null)
  if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !seq_lens || !token_offsets || !workspace || !out)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) || !aligned16(v_scales) ||
      !aligned16(workspace) || !aligned16(out) || (reinterpret_cast<uintptr_t>(flags) & 3u))
    return KVQ_ERR_INVALID_ARG;
  if (!page_table && (int64_t)batch * max_pages > desc->num_pages) return KVQ_ERR_INVALID_ARG;
  if (workspace_bytes < kvq_prompt_workspace_size(desc, n_tokens, num_q_heads, batch, max_seq_len))
    return KVQ_ERR_WORKSPACE;
  const RowsPlan p = plan_prompt(desc, n_tokens, num_q_heads, batch, max_seq_len);
  const bool merge = needs_merge(desc, p);
  RowsArgs r{};
  const OwnArgs own{};
  r.desc = *desc;
  r.q = q;
  r.n_tokens = n_tokens;
  r.num_q_heads = num_q_heads;
  r.group = num_q_heads / desc->num_kv_heads;
  r.k_codes = k_codes;
  r.k_scales = k_scales;
  r.v_codes = v_codes;
  r.v_scales = v_scales;
  r.table = page_table;
  r.max_pages = max_pages;
  r.lens = seq_lens;
  r.max_len = max_seq_len;
  r.offsets = token_offsets;
  r.num_groups = batch;
  r.causal = causal;
  r.sm_scale = sm_scale;
  r.splits = p.splits;
  r.min_chunk = p.min_chunk;
  r.ctas = p.ctas;
  r.chunk_out = static_cast<int32_t*>(workspace) + kChunkWord;
  r.row_tiles = p.row_tiles;
  r.flags = flags ? flags : static_cast<uint32_t*>(workspace);
  if (merge) set_partials(&r, static_cast<uint8_t*>(workspace) + kWorkspaceHeader);
  else r.out = out;
  r.out_f16 = out_type == KVQ_OUT_F16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = launch_rows(r, own, s);
  if (st != KVQ_OK || !merge) return st;
  return launch_rows_merge(r, own, out, r.out_f16, s);
}

int prefix_attn(const kvq_cache_desc* desc, const void* q, int32_t batch, int32_t num_q_heads,
                const void* k_codes, const void* k_scales, const void* v_codes,
                const void* v_scales, const int32_t* prefix_table, int32_t max_prefix_pages,
                const int32_t* prefix_lens, int32_t max_prefix_len,
                const int32_t* group_offsets, int32_t num_groups, const int32_t* page_table,
                int32_t max_pages, const int32_t* seq_lens, int32_t max_seq_len, float sm_scale,
                void* workspace, size_t workspace_bytes, void* out, int32_t out_type,
                uint32_t* flags, void* stream) {
  int st = check_rows(desc, batch, num_q_heads, num_groups, max_prefix_len);
  if (st != KVQ_OK) return st;
  if (max_prefix_pages < 1 || max_pages < 1 || max_seq_len < 0 || num_groups < 1 ||
      (out_type != KVQ_OUT_F32 && out_type != KVQ_OUT_F16) || !isfinite(sm_scale))
    return KVQ_ERR_INVALID_ARG;
  if (batch > KVQ_MAX_BATCH || max_seq_len > kMaxLen) return KVQ_ERR_UNSUPPORTED;
  if (batch == 0) return KVQ_OK;  // (buffers of no elements may be null)
  if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !prefix_lens || !seq_lens || !workspace || !out)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) || !aligned16(v_scales) ||
      !aligned16(workspace) || !aligned16(out) || (reinterpret_cast<uintptr_t>(flags) & 3u))
    return KVQ_ERR_INVALID_ARG;
  if (!group_offsets && num_groups != 1) return KVQ_ERR_INVALID_ARG;
  if (!prefix_table && (int64_t)num_groups * max_prefix_pages > desc->num_pages) return KVQ_ERR_INVALID_ARG;
  if (!page_table && (int64_t)batch * max_pages > desc->num_pages) return KVQ_ERR_INVALID_ARG;
  if (workspace_bytes < kvq_prefix_workspace_size(desc, batch, num_q_heads, num_groups, max_prefix_len, max_seq_len))
    return KVQ_ERR_WORKSPACE;
  const PrefixPlan p = plan_prefix(desc, batch, num_q_heads, num_groups, max_prefix_len, max_seq_len);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  RowsArgs r{};
  r.desc = *desc;
  r.q = q;
  r.n_tokens = batch;
  r.num_q_heads = num_q_heads;
  r.group = num_q_heads / desc->num_kv_heads;
  r.k_codes = k_codes;
  r.k_scales = k_scales;
  r.v_codes = v_codes;
  r.v_scales = v_scales;
  r.table = prefix_table;
  r.max_pages = max_prefix_pages;
  r.lens = prefix_lens;
  r.max_len = max_prefix_len;
  r.offsets = group_offsets;
  r.num_groups = num_groups;
  r.causal = 0;
  r.sm_scale = sm_scale;
  r.splits = p.rows.splits;
  r.min_chunk = p.rows.min_chunk;
  r.ctas = p.rows.ctas;
  r.chunk_out = static_cast<int32_t*>(workspace) + kChunkWord;
  r.row_tiles = max_prefix_len > 0 ? p.rows.row_tiles : 0;
  r.flags = flags ? flags : reinterpret_cast<uint32_t*>(ws);
  set_partials(&r, ws + kWorkspaceHeader);
  OwnArgs own{};
  own.max_splits = p.own_splits;
  own.units = (int64_t)batch * desc->num_kv_heads * p.own_splits;
  own.table = page_table;
  own.max_pages = max_pages;
  own.seq_lens = seq_lens;
  own.max_seq_len = max_seq_len;
  own.split = p.own_split;
  const size_t n_own = (size_t)batch * num_q_heads * p.own_splits;
  own.part_o = reinterpret_cast<float*>(
      ws + kWorkspaceHeader + round256(rows_partial_bytes(batch, num_q_heads, desc->head_dim, p.rows.splits)));
  own.part_m = own.part_o + n_own * desc->head_dim;
  own.part_l = own.part_m + n_own;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (r.row_tiles == 0 || own.units == 0) {
    check_kernel<<<1, 256, 0, s>>>(r, own);
    if (cudaGetLastError() != cudaSuccess) return KVQ_ERR_CUDA;
  }
  st = launch_rows(r, own, s);
  if (st != KVQ_OK) return st;
  return launch_rows_merge(r, own, out, out_type == KVQ_OUT_F16, s);
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

int kvq_plan_step(int32_t batch, int32_t page_size, int32_t num_pages, int32_t max_pages,
                  int32_t max_tokens, const int32_t* seq_lens, const int32_t* new_lens,
                  int32_t* free_pages, const int32_t* free_count, int32_t* page_table,
                  int32_t* seq_lens_out, int32_t* free_count_out, int32_t* token_offsets,
                  int32_t* slots, int32_t* positions, void* workspace, size_t workspace_bytes,
                  void* stream) {
  if (batch < 0 || num_pages < 1 || max_pages < 1 || max_tokens < 0) return KVQ_ERR_INVALID_ARG;
  if (page_size < 64 || page_size % 64 != 0) return KVQ_ERR_UNSUPPORTED;
  if (batch > KVQ_MAX_BATCH || (int64_t)num_pages * page_size > 0x7fffffffLL ||
      (int64_t)max_pages * page_size > 0x7fffffffLL)
    return KVQ_ERR_UNSUPPORTED;
  if (batch == 0) return KVQ_OK;  // (buffers of no elements may be null)
  if (!seq_lens || !new_lens || !free_pages || !free_count || !page_table || !seq_lens_out || !free_count_out ||
      !token_offsets || (!slots && max_tokens > 0) || !workspace)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(slots) || !aligned16(positions) || !aligned16(workspace)) return KVQ_ERR_INVALID_ARG;
  if (workspace_bytes < kWorkspaceHeader) return KVQ_ERR_WORKSPACE;
  PlanArgs a;
  a.batch = batch;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.max_tokens = max_tokens;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.page_table = page_table;
  a.seq_lens_out = seq_lens_out;
  a.free_count_out = free_count_out;
  a.token_offsets = token_offsets;
  a.slots = slots;
  a.positions = positions;
  a.flags = static_cast<uint32_t*>(workspace);
  return launch_plan(a, static_cast<cudaStream_t>(stream));
}

size_t kvq_prompt_workspace_size(const kvq_cache_desc* desc, int32_t n_tokens, int32_t num_q_heads,
                                 int32_t batch, int32_t max_seq_len) {
  if (check_rows(desc, n_tokens, num_q_heads, batch, max_seq_len) != KVQ_OK) return 0;
  const RowsPlan p = plan_prompt(desc, n_tokens, num_q_heads, batch, max_seq_len);
  return kWorkspaceHeader +
         (needs_merge(desc, p) ? rows_partial_bytes(n_tokens, num_q_heads, desc->head_dim, p.splits) : 0);
}

size_t kvq_prefix_workspace_size(const kvq_cache_desc* desc, int32_t batch, int32_t num_q_heads,
                                 int32_t num_groups, int32_t max_prefix_len, int32_t max_seq_len) {
  if (check_rows(desc, batch, num_q_heads, num_groups, max_prefix_len) != KVQ_OK) return 0;
  if (batch > KVQ_MAX_BATCH || max_seq_len < 0 || max_seq_len > kMaxLen) return 0;
  const PrefixPlan p = plan_prefix(desc, batch, num_q_heads, num_groups, max_prefix_len, max_seq_len);
  return kWorkspaceHeader + round256(rows_partial_bytes(batch, num_q_heads, desc->head_dim, p.rows.splits)) +
         rows_partial_bytes(batch, num_q_heads, desc->head_dim, p.own_splits);
}

int kvq_prompt_attn(const kvq_cache_desc* desc, const void* q, int32_t n_tokens,
                    int32_t num_q_heads, const void* k_codes, const void* k_scales,
                    const void* v_codes, const void* v_scales, const int32_t* page_table,
                    int32_t max_pages, const int32_t* seq_lens, int32_t max_seq_len,
                    const int32_t* token_offsets, int32_t batch, int32_t causal, float sm_scale,
                    void* workspace, size_t workspace_bytes, void* out, int32_t out_type,
                    void* stream) {
  return prompt_attn(desc, q, n_tokens, num_q_heads, k_codes, k_scales, v_codes, v_scales, page_table, max_pages, seq_lens,
                     max_seq_len, token_offsets, batch, causal, sm_scale, workspace, workspace_bytes, out, out_type,
                     nullptr, stream);
}

int kvq_prefix_attn(const kvq_cache_desc* desc, const void* q, int32_t batch, int32_t num_q_heads,
                    const void* k_codes, const void* k_scales, const void* v_codes,
                    const void* v_scales, const int32_t* prefix_table, int32_t max_prefix_pages,
                    const int32_t* prefix_lens, int32_t max_prefix_len,
                    const int32_t* group_offsets, int32_t num_groups, const int32_t* page_table,
                    int32_t max_pages, const int32_t* seq_lens, int32_t max_seq_len, float sm_scale,
                    void* workspace, size_t workspace_bytes, void* out, int32_t out_type,
                    void* stream) {
  return prefix_attn(desc, q, batch, num_q_heads, k_codes, k_scales, v_codes, v_scales, prefix_table, max_prefix_pages,
                     prefix_lens, max_prefix_len, group_offsets, num_groups, page_table, max_pages, seq_lens, max_seq_len,
                     sm_scale, workspace, workspace_bytes, out, out_type, nullptr, stream);
}

int kvq_packed_call(int32_t which, const int64_t* w) {
  if (!w) return KVQ_ERR_INVALID_ARG;
  auto ptr = [&](int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(w[i])); };
  auto ints = [&](int i) { return static_cast<int32_t*>(ptr(i)); };
  auto num = [&](int i) { return static_cast<int32_t>(w[i]); };
  auto real = [&](int i) {
    double d;
    memcpy(&d, w + i, sizeof d);
    return static_cast<float>(d);
  };
  const kvq_cache_desc* desc = static_cast<const kvq_cache_desc*>(ptr(0));
  switch (which) {
    case 0:
      return kvq_plan_step(num(0), num(1), num(2), num(3), num(4), ints(5), ints(6), ints(7), ints(8), ints(9), ints(10),
                           ints(11), ints(12), ints(13), ints(14), ptr(15), (size_t)w[16], ptr(17));
    case 1:
      return prompt_attn(desc, ptr(1), num(2), num(3), ptr(4), ptr(5), ptr(6), ptr(7), ints(8), num(9), ints(10),
                         num(11), ints(12), num(13), num(14), real(15), ptr(16), (size_t)w[17], ptr(18), num(19),
                         static_cast<uint32_t*>(ptr(21)), ptr(20));
    case 2:
      return prefix_attn(desc, ptr(1), num(2), num(3), ptr(4), ptr(5), ptr(6), ptr(7), ints(8), num(9), ints(10),
                         num(11), ints(12), num(13), ints(14), num(15), ints(16), num(17), real(18), ptr(19),
                         (size_t)w[20], ptr(21), num(22), static_cast<uint32_t*>(ptr(24)), ptr(23));
    default:
      return KVQ_ERR_INVALID_ARG;
  }
}

}  // extern "C"
