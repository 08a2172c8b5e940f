// One serving step's page bookkeeping (kvq_plan_step): pages of ended requests go back on the
// stack of free pages, the pages that the new tokens need come off it, and every new token gets
// its slot and position.
//
// One thread-block cluster (one CTA when the step is small): every CTA loads all lengths and
// runs the same prefix sums, one thread per request, so that no CTA waits for another's
// result; the pages are then dealt over the cluster.  Bound by latency: a few dependent reads
// and three cluster barriers, which stand between the last read of a buffer and its first write
// (in-place updates) and between the pushes and the pops.  The slots of a small step are written
// by the same CTAs, those of a large one by a second launch over the whole device.
#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_plan.h"

namespace kvq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;
constexpr int64_t kSmallStep = 8192;   // slots that one CTA writes by itself
constexpr int64_t kLargeStep = 65536;  // more slots than this: a second launch over the whole device
static_assert(KVQ_MAX_BATCH <= kPlanThreads, "one thread per request");

struct PlanShared {
  int old_len[KVQ_MAX_BATCH];
  int tok[KVQ_MAX_BATCH + 1];   // first new token of each request
  int need[KVQ_MAX_BATCH + 1];  // first new page
  int rel[KVQ_MAX_BATCH + 1];   // first released page
  long long warp_sum[3][32];
  uint32_t bad;  // KVQ_FLAG_* bits this CTA found
};

// Exclusive prefix sums of three values over the block; total: the sums.
__device__ __forceinline__ void scan3(PlanShared& sh, const long long (&x)[3], long long (&before)[3],
                                      long long (&total)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long v = x[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    before[k] = v - x[k];
    if (lane == 31) sh.warp_sum[k][warp] = v;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long v = sh.warp_sum[k][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    total[k] = __shfl_sync(0xffffffffu, v, 31);
    const long long prev = __shfl_sync(0xffffffffu, v, (warp + 31) & 31);
    before[k] += warp ? prev : 0;
  }
}

// The last index i < n with first[i] <= x (first[0] = 0 <= x).
__device__ __forceinline__ int owner(const int* first, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// OR of every CTA's bits; the barrier inside also orders the cluster's global writes before it.
__device__ __forceinline__ uint32_t cluster_or(PlanShared& sh, uint32_t bits, int ctas) {
  if (bits) atomicOr(&sh.bad, bits);
  if (ctas == 1) {
    __syncthreads();
    return sh.bad;
  }
  cluster_sync();
  uint32_t all = 0;
  for (int c = 0; c < ctas; ++c) all |= __float_as_uint(dsmem_ld(dsmem_addr(&sh.bad, c)));
  return all;
}

// Slots and positions of the tokens t0 .. t0 + 3; behind the last token -1 and 0.  tok: first
// token of each request; old_len(b): its positions before the step; page_of(b, i): its i-th page.
template <class OldLen, class PageOf>
__device__ __forceinline__ void write_slots(const PlanArgs& a, int64_t t0, int tokens, const int* tok,
                                            const OldLen& old_len, const PageOf& page_of) {
  int slot[4] = {-1, -1, -1, -1}, pos[4] = {0, 0, 0, 0};
  if (t0 < tokens) {
    int b = owner(tok, a.batch, (int)t0);
    int n_old = old_len(b);
    int page_index = -1, page = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = (int)t0 + k;
      if (t >= tokens) break;
      if (t >= tok[b + 1]) {
        do ++b; while (t >= tok[b + 1]);
        n_old = old_len(b);
        page_index = -1;
      }
      const int p = n_old + t - tok[b];
      const int pi = (int)((unsigned)p / (unsigned)a.page_size);
      if (pi != page_index) {
        page_index = pi;
        page = page_of(b, pi);
      }
      slot[k] = page * a.page_size + (p - pi * a.page_size);
      pos[k] = p;
    }
  }
  if (t0 + 4 <= a.max_tokens) {
    *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    if (a.positions) *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
  } else {
    for (int k = 0; k < 4 && t0 + k < a.max_tokens; ++k) {
      a.slots[t0 + k] = slot[k];
      if (a.positions) a.positions[t0 + k] = pos[k];
    }
  }
}

// apart: the slots are left to slots_kernel.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a, int ctas, int apart) {
  __shared__ PlanShared sh;
  grid_dependents_launch();
  const int tid = threadIdx.x;
  const int rank = ctas > 1 ? (int)cluster_rank() : 0;
  const int ps = a.page_size;
  const int64_t cap = (int64_t)a.max_pages * ps;
  if (tid == 0) sh.bad = 0;
  int n = 0, add = 0;
  const bool mine = tid < a.batch;
  if (mine) {
    n = a.seq_lens[tid];
    add = a.new_lens[tid];
  }
  const int count = *a.free_count;
  uint32_t bits = 0;
  const bool ended = add == -1;
  if (mine && (n < 0 || n > cap || add < -1 || (int64_t)n + add > cap)) bits = KVQ_FLAG_BAD_SEQLEN;
  const bool use = mine && !bits;
  const int had = use ? (int)(((int64_t)n + ps - 1) / ps) : 0;
  const int fresh = use && !ended ? (int)(((int64_t)n + add + ps - 1) / ps) - had : 0;
  long long x[3] = {use && !ended ? add : 0, fresh, use && ended ? had : 0}, before[3], total[3];
  scan3(sh, x, before, total);
  if (count < 0 || total[2] > (long long)a.num_pages - count) bits |= KVQ_FLAG_BAD_PAGE;
  if (total[1] > count + total[2]) bits |= KVQ_FLAG_NO_PAGES;
  if (total[0] > a.max_tokens) bits |= KVQ_FLAG_NO_SLOTS;
  // every CTA sees the same inputs, so it finds the same bits: a block-wide OR is enough here
  bits = __syncthreads_or((bits & KVQ_FLAG_BAD_SEQLEN) != 0) ? bits | KVQ_FLAG_BAD_SEQLEN : bits;
  if (bits == 0) {  // uniform over the block
    if (mine) {
      sh.old_len[tid] = n;
      sh.tok[tid] = (int)before[0];
      sh.need[tid] = (int)before[1];
      sh.rel[tid] = (int)before[2];
    }
    if (tid == 0) {
      sh.tok[a.batch] = (int)total[0];
      sh.need[a.batch] = (int)total[1];
      sh.rel[a.batch] = (int)total[2];
    }
  }
  __syncthreads();
  const int step = ctas * kPlanThreads, at = rank * kPlanThreads + tid;
  uint32_t found = bits;
  if (bits == 0) {
    // push the released pages (above the count: nothing reads them before the pops)
    for (int e = at; e < (int)total[2]; e += step) {
      const int b = owner(sh.rel, a.batch, e);
      const int page = a.page_table[(int64_t)b * a.max_pages + e - sh.rel[b]];
      if (page < 0 || page >= a.num_pages) found |= KVQ_FLAG_BAD_PAGE;
      a.free_pages[count + e] = page;
    }
    // the page that each request's next token continues
    if (rank == 0 && mine && add > 0 && n % ps != 0) {
      const int page = a.page_table[(int64_t)tid * a.max_pages + had - 1];
      if (page < 0 || page >= a.num_pages) found |= KVQ_FLAG_BAD_PAGE;
    }
  }
  bits = cluster_or(sh, found, ctas);
  const int top = count + (int)total[2];  // pages on the stack
  found = 0;
  if (bits == 0) {
    for (int e = at; e < (int)total[1]; e += step) {
      const int page = a.free_pages[top - 1 - e];
      if (page < 0 || page >= a.num_pages) found |= KVQ_FLAG_BAD_PAGE;
    }
  }
  bits = cluster_or(sh, found, ctas);
  if (bits) {
    if (rank == 0 && tid == 0) set_flag(a.flags, bits);
    total[0] = 0;
  } else {
    for (int e = at; e < (int)total[1]; e += step) {
      const int b = owner(sh.need, a.batch, e);
      const int first = (int)(((int64_t)sh.old_len[b] + ps - 1) / ps);
      a.page_table[(int64_t)b * a.max_pages + first + e - sh.need[b]] = a.free_pages[top - 1 - e];
    }
  }
  const int tokens = (int)total[0];
  if (!apart) {
    for (int64_t t0 = (int64_t)at * 4; t0 < a.max_tokens; t0 += (int64_t)step * 4)
      write_slots(a, t0, tokens, sh.tok, [&](int b) { return sh.old_len[b]; },
                  [&](int b, int pi) {
                    const int had_b = (int)(((int64_t)sh.old_len[b] + ps - 1) / ps);
                    return pi < had_b ? a.page_table[(int64_t)b * a.max_pages + pi]
                                      : a.free_pages[top - 1 - (sh.need[b] + pi - had_b)];
                  });
  }
  if (rank == 0) {
    if (mine) {
      a.token_offsets[tid] = bits ? 0 : sh.tok[tid];
      a.seq_lens_out[tid] = bits ? n : ended ? 0 : n + add;
    }
    if (tid == 0) {
      a.token_offsets[a.batch] = tokens;
      *a.free_count_out = bits ? count : top - (int)total[1];
    }
  }
  if (ctas > 1) cluster_sync();  // no CTA leaves while another may still read its bits
}

// The slots and positions of a large step, over the whole device, from what plan_kernel wrote (a
// refused step has no tokens).
constexpr int kSlotThreads = 256;
__global__ void __launch_bounds__(kSlotThreads) slots_kernel(const PlanArgs a) {
  __shared__ int tok[KVQ_MAX_BATCH + 1];
  grid_dependency_wait();
  for (int b = threadIdx.x; b <= a.batch; b += kSlotThreads) tok[b] = a.token_offsets[b];
  __syncthreads();
  const int64_t t0 = ((int64_t)blockIdx.x * kSlotThreads + threadIdx.x) * 4;
  if (t0 >= a.max_tokens) return;
  write_slots(a, t0, tok[a.batch], tok, [&](int b) { return a.seq_lens_out[b] - (tok[b + 1] - tok[b]); },
              [&](int b, int pi) { return a.page_table[(int64_t)b * a.max_pages + pi]; });
}

}  // namespace

int launch_plan(const PlanArgs& a, cudaStream_t stream) {
  // Up to kSmallStep slots one CTA (256 tokens: 7 us), then a cluster of eight (37,000 slots: 12 us),
  // then the cluster for the pages and a second launch, scheduled early, for the slots (494,000
  // slots: 10 us, against 26 by the cluster alone; the launch itself costs the host 5).  Where the
  // two routes cross between 37,000 and 494,000 was not measured.
  const bool apart = (int64_t)a.max_tokens > kLargeStep;
  const int ctas = (int64_t)a.max_tokens > kSmallStep ? kPlanCluster : 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kPlanThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, plan_kernel, a, ctas, (int)apart) != cudaSuccess) return KVQ_ERR_CUDA;
  if (!apart) return KVQ_OK;
  cudaLaunchConfig_t slots = {};
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  slots.gridDim = dim3((unsigned)(((int64_t)a.max_tokens + 4 * kSlotThreads - 1) / (4 * kSlotThreads)), 1, 1);
  slots.blockDim = dim3(kSlotThreads, 1, 1);
  slots.stream = stream;
  slots.attrs = early;
  slots.numAttrs = 1;
  return cudaLaunchKernelEx(&slots, slots_kernel, a) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace kvq
