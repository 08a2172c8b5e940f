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

struct MergeArgs {
  RowsArgs rows;
  OwnArgs own;
  void* out;
  int out_f16;
};

// Add n partials (consecutive in o, m, l) under the maximum M; mine: this lane's m (of partial
// `lane`) of the first 32.
template <int E>
__device__ __forceinline__ void add_partials(const float* __restrict__ o, const float* __restrict__ m,
                                             const float* __restrict__ l, int n, float M, float mine, int lane,
                                             float (&acc)[E], float& den) {
  constexpr int D = 32 * E;
  constexpr int kBatch = 8;  // reads in flight
  for (int base = 0; base < n; base += 32) {
    const int k = min(32, n - base);
    if (base > 0) mine = lane < k ? m[base + lane] : -INFINITY;
    const float w = lane < k ? ex2(mine - M) : 0.f;
    if (lane < k) den = fmaf(w, l[base + lane], den);
    for (int i = 0; i < k; i += kBatch) {
      float v[kBatch][E];
#pragma unroll
      for (int t = 0; t < kBatch; ++t) load_row<E>(o + (int64_t)(base + min(i + t, k - 1)) * D + lane * E, v[t]);
#pragma unroll
      for (int t = 0; t < kBatch; ++t) {
        const float wi = __shfl_sync(0xffffffffu, w, (i + t) & 31);
        if (i + t < k && wi != 0.f) {
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(wi, v[t][e], acc[e]);
        }
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
  // the token's group: the last one whose first token is not behind it (32 candidates at a time)
  int g = 0, first = 0, n = r.n_tokens;
  bool found = r.num_groups > 0;
  if (r.offsets) {
    int lo = 0, hi = r.num_groups;  // offsets[lo] <= token (or lo = 0), the answer in lo .. hi
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32;
      const int at = min(lo + (lane + 1) * step, hi);
      const uint32_t le = __ballot_sync(0xffffffffu, r.offsets[at] <= token);
      const int k = __popc(le);  // the offsets do not decrease
      const int nlo = k == 0 ? lo : min(lo + k * step, hi);
      hi = k == 32 ? hi : min(lo + (k + 1) * step, hi) - 1;
      lo = nlo;
      if (hi < lo) hi = lo;
    }
    g = lo;
    found = g < r.num_groups;
    if (found) {
      first = r.offsets[g];
      n = r.offsets[g + 1] - first;
      found = first >= 0 && token >= first && token < first + n && first + n <= r.n_tokens;
    }
  }
  int lim = 0, ns = 0, no = 0;
  if (found) {
    int len = r.lens[g];
    if (len < 0 || len > r.max_len || len > (int64_t)r.max_pages * r.desc.page_size) len = 0;
    lim = min(len, row_limit(len, n, token - first, r.causal));
  }
  if (a.own.seq_lens) {  // prefix decode
    int len = a.own.seq_lens[token];
    if (len < 0 || len > a.own.max_seq_len || len > (int64_t)a.own.max_pages * r.desc.page_size) len = 0;
    no = (len + a.own.split - 1) / a.own.split;
  }
  grid_dependency_wait();  // the partials and the chunk
  if (!found && !a.own.seq_lens) return;  // a token behind the last request: left as it was
  const int chunk = r.splits > 1 ? *reinterpret_cast<volatile int32_t*>(r.chunk_out) : r.min_chunk;
  if (lim > 0) ns = (int)(((int64_t)lim + chunk - 1) / chunk);
  const float* pm = r.part_m + row * r.splits;
  const float* om = a.own.part_m + row * a.own.max_splits;
  const float m0 = lane < ns ? pm[lane] : -INFINITY, m1 = lane < no ? om[lane] : -INFINITY;
  float M = fmaxf(m0, m1);
  for (int i = lane + 32; i < ns; i += 32) M = fmaxf(M, pm[i]);
  for (int i = lane + 32; i < no; i += 32) M = fmaxf(M, om[i]);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[E], den = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const bool empty = M == -INFINITY;
  if (empty) M = 0.f;  // nothing to weigh, but a NaN in a sum still counts
  add_partials<E>(r.part_o + row * r.splits * D, pm, r.part_l + row * r.splits, ns, M, m0, lane, acc, den);
  add_partials<E>(a.own.part_o + row * a.own.max_splits * D, om, a.own.part_l + row * a.own.max_splits, no, M, m1,
                  lane, acc, den);
#pragma unroll
  for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  const float inv = row_scale(den, empty);
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

int launch_rows_merge(const RowsArgs& r, const OwnArgs& own, void* out, int out_f16, cudaStream_t stream) {
  const int64_t rows = (int64_t)r.n_tokens * r.num_q_heads;
  if (rows <= 0) return KVQ_OK;
  const int64_t blocks = (rows + kMergeWarps - 1) / kMergeWarps;
  if (blocks > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  const MergeArgs a{r, own, out, out_f16};
  // scheduled while the rows launch still runs; it waits for it on the device
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3(32 * kMergeWarps, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool rot = r.desc.fmt == KVQ_FMT_LUT4;
  const cudaError_t st = r.desc.head_dim == 128 ? (rot ? cudaLaunchKernelEx(&cfg, merge_kernel<128, true>, a)
                                                       : cudaLaunchKernelEx(&cfg, merge_kernel<128, false>, a))
                                                : (rot ? cudaLaunchKernelEx(&cfg, merge_kernel<64, true>, a)
                                                       : cudaLaunchKernelEx(&cfg, merge_kernel<64, false>, a));
  return st == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace kvq
