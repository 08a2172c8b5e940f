// Merge of attention partials into normalized rows: the splits of a rows launch (prompt or
// shared prefix) and, for prefix decode, the splits of each request's own positions.
//   M = max m_s,  out = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s
// One warp per (token, query head); lane l holds D/32 consecutive elements, so a partial is
// one coalesced read.  lut4 rows are rotated back: out = signs .* (1/sqrt(D)) H out'.
#include "kvq_decode_common.cuh"
#include "kvq_rows.h"

namespace kvq {
namespace {

constexpr int kMergeWarps = 4;

template <int E>
__device__ __forceinline__ void load_row(const float* p, float (&v)[E]) {
  if constexpr (E == 4) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x; v[1] = x.y;
  }
}

// Add n partials (consecutive in o, m, l) under the maximum M.
template <int E>
__device__ __forceinline__ void add_partials(const float* __restrict__ o, const float* __restrict__ m,
                                             const float* __restrict__ l, int n, float M, int lane,
                                             float (&acc)[E], float& den) {
  constexpr int D = 32 * E;
  for (int base = 0; base < n; base += 32) {
    const int k = min(32, n - base);
    const float w = lane < k ? ex2(m[base + lane] - M) : 0.f;
    if (lane < k) den = fmaf(w, l[base + lane], den);
#pragma unroll 4
    for (int i = 0; i < k; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      float v[E];
      load_row<E>(o + (int64_t)(base + i) * D + lane * E, v);
      if (wi != 0.f) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wi, v[e], acc[e]);
      }
    }
  }
}

template <int D, bool ROT>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(const MergeArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  const RowsArgs& r = a.rows;
  if (row >= (int64_t)r.n_tokens * r.num_q_heads) return;
  const int token = (int)(row / r.num_q_heads);
  // the token's group: the last one whose first token is not behind it
  int g = 0, first = 0, n = r.n_tokens;
  bool found = r.num_groups > 0;
  if (r.offsets) {
    int lo = 0, hi = r.num_groups;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (r.offsets[mid] <= token) lo = mid; else hi = mid - 1;
    }
    g = lo;
    found = g < r.num_groups;
    if (found) {
      first = r.offsets[g];
      n = r.offsets[g + 1] - first;
      found = first >= 0 && token >= first && token < first + n && first + n <= r.n_tokens;
    }
  }
  if (!found && !a.seq_lens) return;  // a token behind the last request: left as it was
  int ns = 0;
  if (found) {
    int len = r.lens[g];
    if (len < 0 || len > r.max_len || len > (int64_t)r.max_pages * r.desc.page_size) len = 0;
    const int lim = min(len, row_limit(len, n, token - first, r.causal));
    ns = (int)(((int64_t)lim + r.chunk - 1) / r.chunk);
  }
  int no = 0;
  if (a.seq_lens) {
    const int len = max(0, min(a.seq_lens[token], a.max_seq_len));
    no = (len + a.split_tokens - 1) / a.split_tokens;
  }
  const float* pm = r.part_m + row * r.splits;
  const float* om = a.own_m + row * a.max_splits;
  float M = -INFINITY;
  for (int i = lane; i < ns; i += 32) M = fmaxf(M, pm[i]);
  for (int i = lane; i < no; i += 32) M = fmaxf(M, om[i]);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[E], den = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (M != -INFINITY) {
    add_partials<E>(r.part_o + row * r.splits * D, pm, r.part_l + row * r.splits, ns, M, lane, acc, den);
    add_partials<E>(a.own_o + row * a.max_splits * D, om, a.own_l + row * a.max_splits, no, M, lane, acc, den);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] *= inv;
  if constexpr (ROT) {
#pragma unroll
    for (int h = 1; h < E; h <<= 1)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (!(e & h)) {
          const float u = acc[e], v = acc[e + h];
          acc[e] = u + v;
          acc[e + h] = u - v;
        }
#pragma unroll
    for (int b = 1; b < 32; b <<= 1)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float o = __shfl_xor_sync(0xffffffffu, acc[e], b);
        acc[e] = (lane & b) ? o - acc[e] : acc[e] + o;
      }
    const float cs = D == 64 ? 0.125f : 0.08838834764831845f;  // 1/sqrt(D)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= cs * (float)r.desc.signs[lane * E + e];
  }
  if (a.out_f16) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__half*>(a.out) + row * D + lane * E);
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_h2(acc[0], acc[1]), pack_h2(acc[2], acc[3]));
    else
      dst[0] = pack_h2(acc[0], acc[1]);
  } else {
    float* dst = static_cast<float*>(a.out) + row * D + lane * E;
    if constexpr (E == 4)
      *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    else
      *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
  }
}

}  // namespace

int launch_rows_merge(const MergeArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.rows.n_tokens * a.rows.num_q_heads;
  if (rows <= 0) return KVQ_OK;
  const int64_t blocks = (rows + kMergeWarps - 1) / kMergeWarps;
  if (blocks > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  const bool rot = a.rows.desc.fmt == KVQ_FMT_LUT4;
  const unsigned n = (unsigned)blocks;
  if (a.rows.desc.head_dim == 128) {
    if (rot) merge_kernel<128, true><<<n, 32 * kMergeWarps, 0, stream>>>(a);
    else merge_kernel<128, false><<<n, 32 * kMergeWarps, 0, stream>>>(a);
  } else {
    if (rot) merge_kernel<64, true><<<n, 32 * kMergeWarps, 0, stream>>>(a);
    else merge_kernel<64, false><<<n, 32 * kMergeWarps, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace kvq
