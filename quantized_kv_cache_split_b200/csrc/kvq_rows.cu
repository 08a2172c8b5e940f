// Attention of many query rows over the quantized cache (sm_100a): prompt attention (the
// new tokens of each request over its own positions) and the shared part of prefix decode
// (the tokens of every request of a group over the group's prefix).
//
//   S = Q K^T,  P = 2^(S sm_scale log2(e) - m),  O = P V,  l = sum P
//
// with the running maximum m of a streaming softmax, one pass over the positions.  Both
// products run on the fifth-generation tensor cores.  One CTA per unit:
// (group, KV head, 256 query rows, split of the positions).
//
//   warps 0-3, 4-7   softmax of row tile 0 / 1 (stream 0 / 1): one thread per row.  Scores
//                    come from TMEM, weights go back to TMEM as fp16 (the A operand of P V)
//                    over the scores.  The maximum is raised, and the accumulator rescaled,
//                    only when weights may leave fp16: until then they stay below 2^15.
//   warps 8-15       dequantize K and V tiles of 128 positions to fp16 in shared memory, four
//                    warps per half tile.
//   warp 16          issues the MMAs.
//   warp 17          copies the codes and scales of half tiles (64 positions: one contiguous
//                    range of a page) into a ring of staging buffers, ahead of the dequantizers.
//
// A unit of more than 128 rows runs its two row tiles against the same K / V tiles, so a
// tile is dequantized once for 256 rows.  A unit of at most 128 rows gives both streams
// the same rows and every other tile each; the streams' results are merged at the end.
//
// Own positions of prefix decode are units of one warp (kvq_own.cuh) in blocks of the same grid.
//
// Roundings: K and V values to fp16 once (2^-11 relative, as code * scale), the lut4 query after
// its rotation to fp16, the weights to fp16: the operand types of the tensor core.  Scores, maxima,
// sums and accumulators are fp32.
//
// What bounds it.  256 rows x 128 positions at head_dim 128: the MMAs alone 2048 clocks, the
// exponentials alone 2048 (16 a clock and SM), shared memory about 2600 (the fp16 tiles written
// and read by the MMAs, the query read again for every tile, the staged codes); measured 3900.
// Both streams alternate: one's weights are computed while the other's MMAs run.  Measured on a
// 64K q8_0 prefix for 256 requests (32/4 heads, 275 GFLOP): 332 to 340 us back to back, 810 to 830
// TFLOP/s, at 1807 MHz under the power cap; tensor pipe 55 % busy on the SMs at work, exponentials
// 56 %, issue slots 60 %.  Tried and slower there, when a single launch took 291: 64-position tiles
// with two score buffers per stream (345 us), two threads per row (370, register spills), a quarter
// of the exponentials on the FMA pipe (358), a pass for the tile's maximum (321).
// 128 rows or fewer: 2550 clocks for 128 positions, bound by dequantizing through shared memory.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "kvq_own.cuh"
#include "kvq_rows.h"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kSoftmaxWarps = 8, kFillWarps = 8;
constexpr int kMmaWarp = kSoftmaxWarps + kFillWarps, kCopyWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 4);  // a whole warpgroup for the MMA warp
// Registers per thread by role, out of 96 x 640 at launch
constexpr int kSoftmaxRegs = 160, kFillRegs = 64, kMmaRegs = 32;
static_assert(32 * (kSoftmaxWarps * kSoftmaxRegs + kFillWarps * kFillRegs + 4 * kMmaRegs) <= 96 * kThreads,
              "register pool");
constexpr int kOwnWarps = 12, kOwnRegs = 136;  // blocks of own units: three warpgroups of five
static_assert(32 * (kOwnWarps * kOwnRegs + (kThreads / 32 - kOwnWarps) * kMmaRegs) <= 96 * kThreads, "register pool");
// Weights are 2^(s - m + 7).  fp16's smallest step is then 2^-31 of the maximum's weight, so that a
// long tail of small weights is not lost to rounding (with one bit of headroom 64K positions 2^-26
// below the maximum, 0.1 % of the sum, vanished from the product while the denominator counted
// them), and its normal range reaches 2^-21 below.  A tile of equal scores sums to 2^14, half of
// kSafeSum; a maximum may grow 2^1 to 2^8 times before it has to be raised.  (That bit less headroom
// costs 1 % of the 8K prompt and 3 % of the ragged ones.)
constexpr float kWeightBits = 7.f;
constexpr float kSafeSum = 32768.f;  // a tile's weights summing to less are all inside fp16
constexpr uint32_t kTmemColumns = 512;
// q8_0 and nvfp4 values enter the products halved (their rounded code * scale can pass the
// largest fp16 value by a step); the factor goes into the score scale and the output.
template <int FMT>
constexpr float kUnhalve = FMT == KVQ_FMT_Q8_0 || FMT == KVQ_FMT_NVFP4 ? 2.f : 1.f;

constexpr int kMaxRaw = 10;
struct Shared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];  // K / V tile slots
  uint64_t s_full[2], p_half[2], p_full[2];  // a stream's scores; first half, rest of its weights
  uint64_t q_full;                                        // query rows
  uint64_t done;                                          // every MMA completed
  // Staged codes and scales of half tiles.  A stage is filled for either half's warps in turn, and
  // a wait by parity must not meet a phase that is not its waiter's: one barrier per half.
  uint64_t raw_full[2][kMaxRaw], raw_empty[kMaxRaw];
  uint32_t tmem;
  int unit[9];  // see find_unit
  float merge_m[128], merge_l[128];
};

template <int FMT, int D>
struct Smem {
  using C = Cfg<FMT, D>;
  static constexpr int kTileBytes = 128 * D * 2;  // 128 rows of D fp16
  static constexpr int kQ = 0;                    // two row tiles
  static constexpr int kK = 2 * kTileBytes;       // two slots
  static constexpr int kV = 4 * kTileBytes;       // two slots
  static constexpr int kRaw = 6 * kTileBytes;     // staged half tiles: 64 code rows, 64 scale rows
  static constexpr int kRawCodes = kTile * C::CROW, kRawScales = kTile * C::SROW;
  static constexpr int kRawBytes = kRawCodes + kRawScales;
  static constexpr int kRoom = 227 * 1024 - 1024 - (int)sizeof(Shared) - kRaw;
  static constexpr int kStages = kRoom / kRawBytes < kMaxRaw ? kRoom / kRawBytes : kMaxRaw;
  // a unit of one row tile leaves the second one's space to more stages
  static constexpr int kExtra = kTileBytes / kRawBytes < kMaxRaw - kStages ? kTileBytes / kRawBytes : kMaxRaw - kStages;
  static constexpr int kBars = kRaw + kStages * kRawBytes;
  static constexpr int kBytes = kBars + (int)sizeof(Shared) + 1024;  // slack: 1024-byte alignment
  static_assert(256 * (D * 4 + 16) <= kRaw && 128 * (D * 4 + 16) <= kV, "room for the results");
  static_assert(kOwnWarps * Own<FMT, D>::kBytes <= kBars, "room for the own units");
  static_assert(kStages >= 3 && kBars % 16 == 0 && kRawCodes % 128 == 0 && kRawScales % 16 == 0, "staging");
};

// Byte offset of 16-byte chunk c of a row in a [128][D] fp16 tile: column groups of 64, 128-byte
// swizzle.
__device__ __forceinline__ uint32_t tile_offset(int row, int c) {
  return (uint32_t)((c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

// ------------------------------------------------------------------ dequantization
// lo (nvfp4): what the scale d leaves of its exact value, so that a product is rounded once.
template <int FMT, int D>
__device__ __forceinline__ uint4 dequant8(uint32_t w0, uint32_t w1, __half2 d, __half2 lo, const Lut& lut) {
  using C = Cfg<FMT, D>;
  uint4 r;
  if constexpr (C::kQ8) {
    // (byte + 128) | fp16(1024) = 1152 + code; halved: exact
    const __half2 half = __half2half2(__ushort_as_half(0x3800));    // 0.5
    const __half2 bias = __half2half2(__ushort_as_half(0xE080));    // -576
    const uint32_t x0 = w0 ^ 0x80808080u, x1 = w1 ^ 0x80808080u;
    auto two = [&](uint32_t x, uint32_t sel) {
      return h2_as_u32(__hmul2(__hfma2(u32_as_h2(prmt(x, 0x64646464u, sel)), half, bias), d));
    };
    r = make_uint4(two(x0, 0x4140u), two(x0, 0x4342u), two(x1, 0x4140u), two(x1, 0x4342u));
  } else if constexpr (C::kQ4) {
    // low nibble as 1024 + n, high nibble (mantissa bits 4..7) as 64 + n; both less 8
    const __half2 bias = u32_as_h2(0x54806408u);  // (1032, 72)
    auto two = [&](uint32_t sel) {
      const uint32_t t = (prmt(w0, 0u, sel) & 0x00F0000Fu) | 0x54006400u;
      return h2_as_u32(__hmul2(__hsub2(u32_as_h2(t), bias), d));
    };
    r = make_uint4(two(0x4040u), two(0x4141u), two(0x4242u), two(0x4343u));
  } else {
    uint32_t L0, H0, L1, H1;
    lut_lookup4(lut, w0, nib_mask_lo(w0), L0, H0);
    lut_lookup4(lut, w0 >> 16, nib_mask_hi(w0), L1, H1);
    auto two = [&](uint32_t x) {
      if constexpr (C::kNv) return h2_as_u32(__hfma2(u32_as_h2(x), d, __hmul2(u32_as_h2(x), lo)));
      return hmul2u(x, d);
    };
    r = make_uint4(two(prmt(L0, H0, 0x5140u)), two(prmt(L0, H0, 0x7362u)), two(prmt(L1, H1, 0x5140u)),
                   two(prmt(L1, H1, 0x7362u)));
  }
  return r;
}

// Dequantize a staged half tile (64 rows, those at or past n_valid as zeros) into rows row0 ..
// row0 + 63 of a fp16 tile; 128 threads, 16 code bytes at a time.
template <int FMT, int D>
__device__ __forceinline__ void fill_half(const uint8_t* __restrict__ raw, uint8_t* tile, int row0, int n_valid,
                                          int tid, const Lut& lut) {
  using C = Cfg<FMT, D>;
  constexpr int kChunks = C::CROW / 16;          // 16-byte code chunks of a row
  constexpr int kTasks = kTile * kChunks / 128;  // per thread
  static_assert(kTasks >= 1, "a chunk for every thread");
  const uint8_t* scales = raw + kTile * C::CROW;
  // Row and code chunk of task i: dealt so that eight neighbours read eight different bank
  // groups of the staged codes and write eight different ones of the swizzled tile (whose two
  // column groups coincide modulo the banks): rows next to each other take opposite row halves.
  auto place = [&](int i, int& row, int& j) {
    if constexpr (kChunks == 8) {
      row = 2 * (tid >> 3) + (tid >> 2 & 1) + 32 * (i >> 1);
      j = (tid & 3) + 4 * ((tid >> 2 & 1) ^ (i & 1));
    } else if constexpr (kChunks == 4 && !C::kQ8) {
      row = tid >> 1;
      j = (tid & 1) + 2 * ((tid >> 2 & 1) ^ i);
    } else {
      row = (i * 128 + tid) / kChunks;
      j = tid % kChunks;
    }
  };
  // every load first: the stores below might alias them for all the compiler knows
  uint4 u[kTasks];
  __half2 d[kTasks][C::kNv ? 2 : 1], lo[kTasks][C::kNv ? 2 : 1];
#pragma unroll
  for (int i = 0; i < kTasks; ++i) {
    int row, j;
    place(i, row, j);
    u[i] = *reinterpret_cast<const uint4*>(raw + row * C::CROW + j * 16);
    const bool live = row < n_valid;
    const uint8_t* sp = scales + row * C::SROW;
    if constexpr (C::kNv) {
      const uint32_t e = lds16(sp + 2 * j);
      const float g = *reinterpret_cast<const float*>(sp + D / 16);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float x = live ? e4m3_float(e >> (8 * k) & 0xffu) * g : 0.f;
        d[i][k] = __float2half2_rn(x);
        lo[i][k] = __float2half2_rn(x - __low2float(d[i][k]));
      }
    } else {
      const uint32_t b = lds16(sp + (C::kQ8 ? j >> 1 : C::kQ4 ? j : 0) * 2);
      d[i][0] = __half2half2(__ushort_as_half((unsigned short)(live ? b : 0u)));
    }
  }
#pragma unroll
  for (int i = 0; i < kTasks; ++i) {
    int row, j;
    place(i, row, j);
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
    constexpr int kOut = C::kQ8 ? 2 : 4;  // 16-byte chunks of eight values
#pragma unroll
    for (int c = 0; c < kOut; ++c) {
      const int b = C::kNv ? c >> 1 : 0;
      const uint4 v = C::kQ8 ? dequant8<FMT, D>(w[2 * c & 3], w[(2 * c + 1) & 3], d[i][0], d[i][0], lut)
                             : dequant8<FMT, D>(w[c], 0u, d[i][b], lo[i][b], lut);
      *reinterpret_cast<uint4*>(tile + tile_offset(row0 + row, kOut * j + c)) = v;
    }
  }
}

// ------------------------------------------------------------------ unit lookup
// A group's tokens and positions, checked; the tokens are 0 when they are out of range.
struct Group {
  int first, tokens, len;
};
__device__ __forceinline__ Group read_group(const RowsArgs& a, int g) {
  const int first = a.offsets ? a.offsets[g] : 0, end = a.offsets ? a.offsets[g + 1] : a.n_tokens;
  int len = a.lens[g];
  const bool bad_len = len < 0 || len > a.max_len || len > (int64_t)a.max_pages * a.desc.page_size;
  const bool bad = first < 0 || end < first || end > a.n_tokens;
  if (bad || bad_len) set_flag(a.flags, KVQ_FLAG_BAD_SEQLEN);
  return Group{first, bad ? 0 : end - first, bad_len ? 0 : len};
}

// Block `t`'s unit: group, first row, rows, positions, first token, tokens (0: no such unit), KV
// head, split, positions per split.  One warp.
//
// Up to 32 groups: one per lane, units counted exactly.  The chunk balances groups of unequal
// lengths: about the shortest multiple of kKvTile for which the units (row tile, KV head, split)
// number at most a.ctas.
// More groups: the row tiles of group g (rows s .. e - 1 of all groups' rows) take the slots from
// floor(s / kRowTile) + g, which leaves room for ceil((e - s) / kRowTile) of them, so that a block
// finds its group by a search instead of a sum over all groups.  The chunk is a.min_chunk.
__device__ __forceinline__ void find_unit(const RowsArgs& a, int t, int lane, int* unit) {
  const int hkv = a.desc.num_kv_heads;
  auto tiles_of = [&](int n) { return (n * a.group + kRowTile - 1) / kRowTile; };
  // splits of a group; with direct output a unit without positions still writes its zeros
  auto splits_of = [&](int len, int chunk) { return max((len + chunk - 1) / chunk, a.out ? 1 : 0); };
  auto put = [&](int g, const Group& x, int row_tile, int head, int split, int chunk) {
    // the last rows of a causal group see the most positions: they start first
    const int tile = a.causal ? tiles_of(x.tokens) - 1 - row_tile : row_tile;
    unit[0] = g;
    unit[1] = tile * kRowTile;
    unit[2] = min(x.tokens * a.group - tile * kRowTile, kRowTile);
    unit[3] = x.len;
    unit[4] = x.first;
    unit[5] = x.tokens;
    unit[6] = head;
    unit[7] = split;
    unit[8] = chunk;
  };
  if (lane == 0) unit[5] = 0;
  __syncwarp();
  int chunk = a.min_chunk;
  if (a.num_groups > 32) {
    if (a.splits > 1 && t == 0 && lane == 0) *a.chunk_out = chunk;
    const int split = t % a.splits, head = t / a.splits % hkv, slot = t / a.splits / hkv;
    auto first_slot = [&](int g) { return (int)((int64_t)a.offsets[g] * a.group / kRowTile) + g; };
    int lo = 0, hi = a.num_groups - 1;  // the last group whose first slot is not behind this one
    while (lo < hi) {
      const int step = (hi - lo + 31) >> 5;
      const int k = __popc(__ballot_sync(0xffffffffu, first_slot(min(lo + (lane + 1) * step, hi)) <= slot));
      const int next = min(lo + k * step, hi);
      if (k < 32) hi = max(next, min(lo + (k + 1) * step, hi) - 1);
      lo = next;
    }
    if (lane == 0) {
      const Group x = read_group(a, lo);
      const int row_tile = slot - first_slot(lo);
      if (row_tile >= 0 && row_tile < tiles_of(x.tokens) && split < splits_of(x.len, chunk))
        put(lo, x, row_tile, head, split, chunk);
    }
    __syncwarp();
    return;
  }
  Group x{0, 0, 0};
  if (lane < a.num_groups) x = read_group(a, lane);
  const int tiles = tiles_of(x.tokens);
  if (a.splits > 1) {
    // In tiles of kKvTile.  32 candidates at a time, one per lane, between the even share of all
    // the work and the longest group; then again around the best.  (The candidates' units by
    // approximate reciprocals: a unit more or less than a.ctas only costs balance.)
    const int t0 = tiles * hkv, l0 = (x.len + kKvTile - 1) / kKvTile;
    const float share = (float)__reduce_add_sync(0xffffffffu, (unsigned)(t0 * l0)) / (float)a.ctas;
    int lo = max(max(a.min_chunk / kKvTile, 1), (int)ceilf(share));
    int hi = max(lo, (int)__reduce_max_sync(0xffffffffu, (unsigned)l0));
    for (int pass = 0; pass < 2 && lo < hi; ++pass) {
      const int step = (hi - lo + 31) >> 5;
      const int c = min(lo + lane * step, hi);
      const float r = __frcp_rn((float)c);
      int u = 0;
      for (int g = 0; g < a.num_groups; ++g)
        u += __shfl_sync(0xffffffffu, t0, g) * (int)ceilf((float)__shfl_sync(0xffffffffu, l0, g) * r - 1e-3f);
      const uint32_t fits = __ballot_sync(0xffffffffu, u <= a.ctas);
      const int k = fits ? __ffs(fits) - 1 : 32;
      hi = min(lo + k * step, hi);
      lo = k > 0 ? min(lo + (k - 1) * step + 1, hi) : lo;
    }
    chunk = hi * kKvTile;
    if (t == 0 && lane == 0) *a.chunk_out = chunk;
  }
  const int splits = splits_of(x.len, chunk), mine = tiles * splits * hkv;
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += y;
  }
  before -= mine;
  if (t >= before && t < before + mine) {  // split fastest, then KV head
    const int k = t - before;
    put(lane, x, k / splits / hkv, k / splits % hkv, k % splits, chunk);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ the kernel
template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const RowsArgs a, const OwnArgs own) {
  using C = Cfg<FMT, D>;
  using S = Smem<FMT, D>;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  Shared& sh = *reinterpret_cast<Shared*>(smem + S::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hkv = a.desc.num_kv_heads, G = a.group;
  grid_dependents_launch();  // the merge may be scheduled (it waits for this grid's results)
  // Blocks of own units stand behind the first a.ctas row blocks: those past them have a unit only
  // when no cut of the groups brings the units down to a.ctas.
  const int row_blocks = a.row_tiles * hkv * a.splits, own_blocks = (int)gridDim.x - row_blocks;
  const int own_first = min(row_blocks, a.ctas), own_index = (int)blockIdx.x - own_first;
  if (own_index >= 0 && own_index < own_blocks) {
    // the requests' own positions: twelve warps, a unit each
    if (warp < kOwnWarps) {
      regs_grow<kOwnRegs>();
      const int64_t u = (int64_t)own_index * kOwnWarps + warp;
      if (u < own.units) own_unit<FMT, D>(own, a, u, smem + warp * Own<FMT, D>::kBytes, lane);
    } else {
      regs_shrink<kMmaRegs>();
    }
    return;
  }

  const int block = own_index < 0 ? (int)blockIdx.x : (int)blockIdx.x - own_blocks;
  if (warp == 0) find_unit(a, block, lane, sh.unit);
  // (many groups: the search looks at a few of them; one block checks them all)
  if (warp == kCopyWarp + 1 && block == 0 && a.num_groups > 32)
    for (int g = lane; g < a.num_groups; g += 32) (void)read_group(a, g);
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem, kTmemColumns);
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        bar_init(&sh.k_full[i], kFillWarps);
        bar_init(&sh.v_full[i], kFillWarps);
        bar_init(&sh.k_empty[i], 1);
        bar_init(&sh.v_empty[i], 1);
        bar_init(&sh.s_full[i], 1);
        bar_init(&sh.p_half[i], kSoftmaxWarps / 2);
        bar_init(&sh.p_full[i], kSoftmaxWarps / 2);
      }
      bar_init(&sh.q_full, kSoftmaxWarps);
      bar_init(&sh.done, 1);
      for (int i = 0; i < S::kStages + S::kExtra; ++i) {
        bar_init(&sh.raw_full[0][i], 1);
        bar_init(&sh.raw_full[1][i], 1);
        bar_init(&sh.raw_empty[i], kFillWarps / 2);
      }
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int g = sh.unit[0], row0 = sh.unit[1], rows = sh.unit[2], len = sh.unit[3], tok0 = sh.unit[4], n = sh.unit[5];
  const int kvh = sh.unit[6], split = sh.unit[7], chunk = sh.unit[8];
  // positions of this split that any row of the unit sees
  const int last = n > 0 ? row_limit(len, n, (row0 + rows - 1) / G, a.causal) : 0;
  const int begin = n > 0 ? split * chunk : 0;
  const int end = n > 0 ? min(min(last, len), begin + chunk) : 0;
  const int tiles = end > begin ? (end - begin + kKvTile - 1) / kKvTile : 0;
  const bool shared_tiles = rows > 128;  // both streams take every tile; else every other one
  const bool live = n > 0 && (tiles > 0 || a.out != nullptr);
  // row r of the unit: token tok_base + t, head h of the KV head's G, t = (r + h_base) / G by a 16-bit
  // reciprocal (exact below 8192)
  const int tok_base = row0 / G, h_base = row0 - tok_base * G;
  const uint32_t g_inv = 65536u / (uint32_t)G + 1u;
  auto token_of = [&](int r) { return tok_base + (int)(((uint32_t)(r + h_base) * g_inv) >> 16); };
  auto row_index = [&](int r) {  // in q, the output and the partials
    const int t = token_of(r);
    return (int64_t)(tok0 + t) * a.num_q_heads + kvh * G + (row0 + r - t * G);
  };
  const int stages = shared_tiles ? S::kStages : S::kStages + S::kExtra;
  auto stage_at = [&](int st) {
    return smem + (st < S::kStages ? S::kRaw + st * S::kRawBytes : S::kQ + S::kTileBytes + (st - S::kStages) * S::kRawBytes);
  };

  const uint32_t tmem = sh.tmem;
  bool ok = true;

  if (live && tiles > 0) {
    if (warp >= kMmaWarp) {
      // ---------------------------------------------------------------- MMA
      regs_shrink<kMmaRegs>();
      if (warp == kMmaWarp) {
        // the whole warp walks the loop (so that addresses stay warp-uniform); one elected
        // thread issues
        constexpr uint32_t kIdS = mma_idesc(128, kKvTile, false);
        constexpr uint32_t kIdO = mma_idesc(128, D, true);
        constexpr uint32_t kTileUnits = S::kTileBytes >> 4;  // descriptor addresses count 16 bytes
        const bool leader = elect_one();
        const uint64_t qd = mma_desc(smem_u32(smem + S::kQ), 16, 1024);
        const uint64_t kd = mma_desc(smem_u32(smem + S::kK), 16, 1024);
        const uint64_t vd = mma_desc(smem_u32(smem + S::kV), 16384, 1024);
        auto qk = [&](int s, int slot) {
          const uint64_t qa = qd + (shared_tiles ? s : 0) * kTileUnits, ka = kd + slot * kTileUnits;
          const uint32_t dst = tmem + s * 128;
          if (leader) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (k >> 2) * 1024 + (k & 3) * 2;
              mma_ss(dst, qa + off, ka + off, kIdS, k > 0);
            }
            mma_commit(&sh.s_full[s]);
          }
        };
        // step i of stream s: the first half of the tile's positions as soon as their weights
        // are there
        auto pv = [&](int s, int slot, int i) {
          const uint64_t va = vd + slot * kTileUnits;
          const uint32_t dst = tmem + 256 + s * D, src = tmem + s * 128;
          if (!bar_wait(&sh.p_half[s], i & 1)) return false;
          tc_fence_after();
          if (leader) {
            mma_ts(dst, src, va, kIdO, i > 0);
#pragma unroll
            for (int k = 1; k < kKvTile / 32; ++k) mma_ts(dst, src + k * 8, va + k * 128, kIdO, true);
          }
          if (!bar_wait(&sh.p_full[s], i & 1)) return false;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int k = kKvTile / 32; k < kKvTile / 16; ++k) mma_ts(dst, src + k * 8, va + k * 128, kIdO, true);
          }
          return true;
        };
        auto commit = [&](uint64_t* bar) {
          if (leader) mma_commit(bar);
        };
        ok = bar_wait(&sh.q_full, 0);
        if (shared_tiles) {
          ok = ok && bar_wait(&sh.k_full[0], 0);
          if (ok) {
            tc_fence_after();
            qk(0, 0);
            qk(1, 0);
            commit(&sh.k_empty[0]);
          }
          for (int t = 0; ok && t < tiles; ++t) {
            const int slot = t & 1, next = (t + 1) & 1;
            ok = bar_wait(&sh.v_full[slot], t >> 1 & 1);
            for (int s = 0; ok && s < 2; ++s) {
              ok = pv(s, slot, t);
              if (!ok) break;
              if (s == 1) commit(&sh.v_empty[slot]);
              if (t + 1 < tiles) {
                if (s == 0) {
                  ok = bar_wait(&sh.k_full[next], (t + 1) >> 1 & 1);
                  if (!ok) break;
                  tc_fence_after();
                }
                qk(s, next);
                if (s == 1) commit(&sh.k_empty[next]);
              }
            }
          }
        } else {
          for (int s = 0; ok && s < 2 && s < tiles; ++s) {
            ok = bar_wait(&sh.k_full[s], 0);
            if (!ok) break;
            tc_fence_after();
            qk(s, s);
            commit(&sh.k_empty[s]);
          }
          for (int t = 0; ok && t < tiles; ++t) {
            const int s = t & 1, i = t >> 1;
            ok = bar_wait(&sh.v_full[s], i & 1) && pv(s, s, i);
            if (!ok) break;
            commit(&sh.v_empty[s]);
            if (t + 2 < tiles) {
              ok = bar_wait(&sh.k_full[s], (i + 1) & 1);
              if (!ok) break;
              tc_fence_after();
              qk(s, s);
              commit(&sh.k_empty[s]);
            }
          }
        }
        commit(&sh.done);
      }
      if (warp == kCopyWarp) {
        // -------------------------------------------------------------- copies
        // codes and scales of the tiles in the order of the dequantizers, a half tile (64
        // positions of one page) at a time, as far ahead as the staging ring allows
        const uint8_t* kc = static_cast<const uint8_t*>(a.k_codes);
        const uint8_t* ks = static_cast<const uint8_t*>(a.k_scales);
        const uint8_t* vc = static_cast<const uint8_t*>(a.v_codes);
        const uint8_t* vs = static_cast<const uint8_t*>(a.v_scales);
        const int ps = a.desc.page_size;
        // first cache row of 64-position block hb of the split, -1 for a page out of range
        auto row_of = [&](int hb) -> int {
          const int p = begin + hb * kTile;
          if (p >= end) return -1;
          const int pg = p / ps;
          const int page = a.table ? __ldg(a.table + (int64_t)g * a.max_pages + pg) : g * a.max_pages + pg;
          if (page < 0 || page >= a.desc.num_pages) {
            set_flag(a.flags, KVQ_FLAG_BAD_PAGE);
            return -1;
          }
          return (page * hkv + kvh) * ps + (p - pg * ps);
        };
        int krow = row_of(lane), vrow = krow;  // of blocks 32 i + lane, i the current window
        int h = 0, st = 0;      // half tiles so far, the stage of the next
        uint32_t round = 0u;    // parity of the ring's passes
        uint32_t phase0 = 0u, phase1 = 0u, last = 0u;  // per stage: each half's next parity, the half that used it last
        for (int t = -2; ok && t < tiles; ++t) {
          for (int which = 0; ok && which < 2; ++which) {
            const int tt = which ? t + 2 : t;
            if (tt < 0 || tt >= tiles) continue;
            for (int half = 0; ok && half < 2; ++half) {
              const int hb = 2 * tt + half;
              if (begin + hb * kTile >= end) break;
              if ((hb & 31) == 0 && hb > 0) {
                const int next = row_of(hb + lane);
                if (which) krow = next; else vrow = next;
              }
              const int row = __shfl_sync(0xffffffffu, which ? krow : vrow, hb & 31);
              ok = h < stages || bar_wait(&sh.raw_empty[st], round ^ 1);
              if (!ok) break;
              if (lane == 0) {
                uint8_t* dst = stage_at(st);
                uint64_t* full = &sh.raw_full[half][st];
                if (row >= 0) {
                  bar_expect(full, S::kRawBytes);
                  bulk_load(dst, (which ? kc : vc) + (int64_t)row * C::CROW, S::kRawCodes, full);
                  bulk_load(dst + S::kRawCodes, (which ? ks : vs) + (int64_t)row * C::SROW, S::kRawScales, full);
                } else {
                  bar_arrive(full);  // whatever the stage holds: the call is flagged
                }
              }
              if (half) phase1 ^= 1u << st; else phase0 ^= 1u << st;
              last = (last & ~(1u << st)) | (uint32_t)half << st;
              ++h;
              if (++st == stages) {
                st = 0;
                round ^= 1u;
              }
            }
          }
        }
        // no copy may land after the block has gone (each was waited for, unless a wait gave up)
        for (st = 0; st < min(h, stages); ++st) {
          const int half = last >> st & 1;
          (void)bar_wait(&sh.raw_full[half][st], ((half ? phase1 : phase0) >> st & 1) ^ 1);
        }
      }
      __syncwarp();
    } else if (warp >= kSoftmaxWarps) {
      // ---------------------------------------------------------------- dequantize
      // K0 K1 V0 K2 V1 K3 ...: the order in which the MMAs of either mode need the tiles
      regs_shrink<kFillRegs>();
      const int ft = tid - 32 * kSoftmaxWarps;
      Lut lut;
      if constexpr (C::kLut || C::kNv) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (C::kLut) {
            uint32_t e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) e[k] = a.desc.codebook[4 * i + k];
            lut.lo[i] = (e[0] & 0xffu) | (e[1] & 0xffu) << 8 | (e[2] & 0xffu) << 16 | (e[3] & 0xffu) << 24;
            lut.hi[i] = e[0] >> 8 | (e[1] >> 8) << 8 | (e[2] >> 8) << 16 | (e[3] >> 8) << 24;
          } else {
            // E2M1 values 0 0.5 1 1.5 2 3 4 6 and their negatives, halved: fp16 high bytes
            lut.lo[i] = 0u;
            lut.hi[i] = i == 0 ? 0x3A383400u : i == 1 ? 0x42403E3Cu : i == 2 ? 0xBAB8B480u : 0xC2C0BEBCu;
          }
        }
      }
      // four warps per half tile; a half past the last position is filled with zeros
      const int half = ft >> 7;
      int next_stage = 0;    // of this tile's first half
      uint32_t phase = 0u;   // next parity of this half's barrier of each stage
      auto put = [&](int t, uint8_t* slots, uint64_t* full, uint64_t* empty) {
        const int p = begin + t * kKvTile;
        const int n_half = p + kTile < end ? 2 : 1;
        ok = t < 2 || bar_wait(&empty[t & 1], (t >> 1 & 1) ^ 1);
        if (!ok) return;
        const int st = next_stage + half < stages ? next_stage + half : 0;
        const uint8_t* raw = stage_at(st);
        if (half < n_half) {
          ok = bar_wait(&sh.raw_full[half][st], phase >> st & 1);
          if (!ok) return;
          phase ^= 1u << st;
        }
        fill_half<FMT, D>(raw, slots + (t & 1) * S::kTileBytes, half * kTile, end - p - half * kTile, ft & 127, lut);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&full[t & 1]);
          if (half < n_half) bar_arrive(&sh.raw_empty[st]);
        }
        next_stage += n_half;
        if (next_stage >= stages) next_stage -= stages;
      };
      for (int t = -2; ok && t < tiles; ++t) {
        if (t >= 0) put(t, smem + S::kV, sh.v_full, sh.v_empty);
        if (ok && t + 2 < tiles) put(t + 2, smem + S::kK, sh.k_full, sh.k_empty);
      }
    } else {
      // ---------------------------------------------------------------- softmax
      regs_grow<kSoftmaxRegs>();
      // query rows, fp16, K-major, 128-byte swizzle; rows past the unit's are zero.  The loads
      // of several rows are in flight together.  A unit of one row tile has one for both streams.
      {
        const __half* q = static_cast<const __half*>(a.q);
        const bool zero = a.sm_scale == 0.f;
        const uint32_t flip = a.sm_scale < 0.f ? 0x80008000u : 0u;  // the scale's sign goes into the query
        const int n_rows = shared_tiles ? kRowTile : 128;
        auto src = [&](int r) { return q + row_index(r) * D; };
        if constexpr (!C::kLut) {
          constexpr int kC = D / 8, kStep = 32 * kSoftmaxWarps / kC, kBatch = 16;
          const int c = tid % kC;
          for (int r0 = tid / kC; r0 < n_rows; r0 += kBatch * kStep) {
            uint4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int r = r0 + i * kStep;
              v[i] = make_uint4(0u, 0u, 0u, 0u);
              if (r < rows && !zero) v[i] = __ldg(reinterpret_cast<const uint4*>(src(r)) + c);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int r = r0 + i * kStep;
              if (r >= n_rows) break;
              v[i].x ^= flip; v[i].y ^= flip; v[i].z ^= flip; v[i].w ^= flip;
              uint8_t* dst = smem + S::kQ + (r >> 7) * S::kTileBytes + tile_offset(r & 127, c);
              *reinterpret_cast<uint4*>(dst) = v[i];
            }
          }
        } else {
          // rotated: (1/sqrt(D)) H (signs .* q); D / 16 lanes per row, 16 elements each
          constexpr int kL = D / 16, kR = 32 / kL;  // lanes per row, rows per warp
          const int part = lane % kL;
          float sg[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            sg[k] = (float)a.desc.signs[part * 16 + k] * (D == 64 ? 0.125f : 0.08838834764831845f);
          for (int r = warp * kR + lane / kL; r < n_rows; r += kSoftmaxWarps * kR) {
            uint4 raw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
            if (r < rows && !zero) {
              const uint4* p = reinterpret_cast<const uint4*>(src(r)) + part * 2;
              raw[0] = __ldg(p);
              raw[1] = __ldg(p + 1);
            }
            const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
            float y[16];
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float2 f = __half22float2(u32_as_h2(w[k / 2] ^ flip));
              y[k] = f.x * sg[k];
              y[k + 1] = f.y * sg[k + 1];
            }
#pragma unroll
            for (int h = 1; h < 16; h <<= 1)
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (!(k & h)) {
                  const float u = y[k], x = y[k + h];
                  y[k] = u + x;
                  y[k + h] = u - x;
                }
#pragma unroll
            for (int b = 1; b < kL; b <<= 1) {
              const float sign = (lane & b) ? -1.f : 1.f;
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] = fmaf(y[k], sign, __shfl_xor_sync(0xffffffffu, y[k], b));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float* z = y + 8 * c;
              const uint4 h = make_uint4(pack_h2(z[0], z[1]), pack_h2(z[2], z[3]), pack_h2(z[4], z[5]), pack_h2(z[6], z[7]));
              uint8_t* dst = smem + S::kQ + (r >> 7) * S::kTileBytes + tile_offset(r & 127, part * 2 + c);
              *reinterpret_cast<uint4*>(dst) = h;
            }
          }
        }
        fence_async_shared();
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.q_full);
      const int s = warp >> 2;
      const int r = tid & 127;  // row of the row tile = TMEM lane
      const int rr = shared_tiles ? s * 128 + r : r;
      const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's lanes
      const float scale = (a.sm_scale == 0.f ? 1.f : fabsf(a.sm_scale)) * kLog2e * kUnhalve<FMT>;
      const int limit = rr < rows ? min(row_limit(len, n, token_of(rr), a.causal), end) : end;
      const int steps = shared_tiles ? tiles : (tiles - s + 1) / 2;
      const uint32_t ts = at + s * 128, to = at + 256 + s * D;  // scores, accumulator
      const uint64_t scale2 = pack_f2(scale, scale);
      const bool idle = (shared_tiles ? s * 128 : 0) + (warp & 3) * 32 >= rows;  // no row of this warp exists
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < steps; ++i) {
        const int t = shared_tiles ? i : 2 * i + s;
        const int lim = limit - begin - t * kKvTile;  // visible columns of this row in the tile
        ok = bar_wait(&sh.s_full[s], i & 1);
        if (!ok) break;
        tc_fence_after();
        if (idle) {  // the MMA reads whatever these rows hold: rows do not mix
          if (lane == 0) {
            bar_arrive(&sh.p_half[s]);
            bar_arrive(&sh.p_full[s]);
          }
          continue;
        }
        const bool mask = __any_sync(0xffffffffu, lim < kKvTile);
        // No pass over the tile for its maximum: the weights are taken under the maximum that
        // was last raised, and their sum (which the denominator needs anyway) tells whether one
        // may have outgrown fp16: below 2^15 none has.  A maximum 2^8 times the old one always
        // gets there, one that is not above it never does.  Then, and on a row's first
        // positions, the maximum is raised and the tile done again.
        bool raise = __any_sync(0xffffffffu, m == -INFINITY && lim > 0);
        float l0, l1;
        uint32_t p[kKvTile / 2];
        for (;;) {
          float v[2][32];
          auto load = [&](int c, float* x) { tmem_ld32(ts + c * 32, x); };
          auto ready = [&](int c, float* x) {
            tmem_wait_ld32(x);
            if (mask) {
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = c * 32 + k < lim ? x[k] : -INFINITY;
            }
          };
          if (raise) {
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
            for (int c = 0; c < kKvTile / 32; c += 2) {
              load(c, v[0]);
              load(c + 1, v[1]);
              ready(c, v[0]);
              ready(c + 1, v[1]);
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                mx[0] = max3(mx[0], v[0][k], v[0][k + 1]);
                mx[1] = max3(mx[1], v[1][k], v[1][k + 1]);
              }
            }
            const float tm = fmaxf(mx[0], mx[1]) * scale;
            const float f = tm > m ? ex2(m - tm) : 1.f;  // m = -inf: 0
            m = fmaxf(m, tm);
            l *= f;
            // the scores of this tile were issued after the last P V of this stream, so the
            // accumulator is at rest
            if (i > 0) {
#pragma unroll 1
              for (int c = 0; c < D; c += 8) {
                float o[8];
                tmem_ld8(to + c, o);
                tmem_wait_ld8(o);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] *= f;
                tmem_st8(to + c, o);
              }
              tmem_wait_st();
            }
          }
          const float off = m == -INFINITY ? 0.f : kWeightBits - m;
          const uint64_t off2 = pack_f2(off, off);
          uint64_t sum[2] = {0ull, 0ull};  // pairs of fp32 zeros
          load(0, v[0]);
#pragma unroll
          for (int c = 0; c < kKvTile / 32; ++c) {
            float* x = v[c & 1];
            ready(c, x);
            if (c + 1 < kKvTile / 32) load(c + 1, v[(c + 1) & 1]);
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const uint64_t y = fma_f2(pack_f2(x[k], x[k + 1]), scale2, off2);
              float e0, e1;
              unpack_f2(y, e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              sum[(k >> 1) & 1] = add_f2(sum[(k >> 1) & 1], pack_f2(e0, e1));
              p[c * 16 + (k >> 1)] = pack_h2(e0, e1);
            }
          }
          unpack_f2(add_f2(sum[0], sum[1]), l0, l1);
          if (raise || !__any_sync(0xffffffffu, l0 + l1 >= kSafeSum)) break;
          raise = true;
        }
        tmem_st16(ts, p);
        tmem_st16(ts + 16, p + 16);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.p_half[s]);
        tmem_st16(ts + 32, p + 32);
        tmem_st16(ts + 48, p + 48);
        l += l0 + l1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.p_full[s]);
      }
      if (ok) ok = bar_wait(&sh.done, 0);
      tc_fence_after();
      // ---------------------------------------------------------------- results
      m -= kWeightBits;  // of the weights
      const float vscale = kUnhalve<FMT>;
      float f0 = vscale, f1 = 0.f;
      float4* stage = reinterpret_cast<float4*>(smem + S::kV) + r;  // [D / 4][128], stream 1's rows
      if (!shared_tiles) {
        // streams 0 and 1 hold the same rows: stream 1 hands its sums to stream 0
        if (s == 1) {
          sh.merge_m[r] = m;
          sh.merge_l[r] = l;
          if (steps > 0) {
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              float v[32];
              tmem_ld32(to + c, v);
              tmem_wait_ld32(v);
#pragma unroll
              for (int k = 0; k < 32; k += 4)
                stage[(c + k) / 4 * 128] = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            }
          }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (s == 0) {
          const float m1 = sh.merge_m[r], l1 = sh.merge_l[r];
          const float mm = fmaxf(m, m1);
          const float e0 = mm == -INFINITY ? 0.f : ex2(m - mm), e1 = mm == -INFINITY ? 0.f : ex2(m1 - mm);
          l = l * e0 + l1 * e1;
          m = mm;
          f0 = e0 * vscale;
          f1 = tiles > 1 ? e1 * vscale : 0.f;
        }
      }
      // every lane takes part in the TMEM loads; rows past the unit's are not written
      if (shared_tiles || s == 0) {
        const bool write = ok && rr < rows, half = a.out && a.out_f16;
        const int64_t row = write ? row_index(rr) : 0;
        const int64_t part = row * a.splits + split;
        // every tile has been read: the query and K / V space holds the rows (16 bytes of
        // padding between them), each copied out by the thread that owns it
        uint8_t* mine = smem + S::kQ + (s * 128 + r) * (D * 4 + 16);
        if (a.out) {
          const float inv = row_scale(l, m == -INFINITY);
          f0 *= inv;
          f1 *= inv;
        } else if (write) {
          a.part_m[part] = m;
          a.part_l[part] = l;
        }
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(to + c, v);
          tmem_wait_ld32(v);
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float4 o = make_float4(v[k] * f0, v[k + 1] * f0, v[k + 2] * f0, v[k + 3] * f0);
            if (f1 != 0.f) {
              const float4 x = stage[(c + k) / 4 * 128];
              o.x = fmaf(x.x, f1, o.x); o.y = fmaf(x.y, f1, o.y);
              o.z = fmaf(x.z, f1, o.z); o.w = fmaf(x.w, f1, o.w);
            }
            if (half)
              *reinterpret_cast<uint2*>(mine + (c + k) * 2) = make_uint2(pack_h2(o.x, o.y), pack_h2(o.z, o.w));
            else
              *reinterpret_cast<float4*>(mine + (c + k) * 4) = o;
          }
        }
        fence_async_shared();
        if (write) {
          uint8_t* dst = half    ? static_cast<uint8_t*>(a.out) + row * D * 2
                         : a.out ? static_cast<uint8_t*>(a.out) + row * D * 4
                                 : reinterpret_cast<uint8_t*>(a.part_o + part * D);
          bulk_store(dst, mine, half ? D * 2 : D * 4);
          bulk_store_wait();
        }
      }
    }
  } else if (live && warp < kSoftmaxWarps && tid < rows) {
    // no position at all: the rows are zero
    const int64_t row = row_index(tid);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + row * D * (a.out_f16 ? 2 : 4));
    for (int k = 0; k < D * (a.out_f16 ? 2 : 4) / 16; ++k) dst[k] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (!ok) set_flag(a.flags, KVQ_FLAG_TIMEOUT);
  // the MMAs still in flight (after a wait that gave up) end before the TMEM is freed
  if (warp == kMmaWarp && live && tiles > 0) (void)bar_wait(&sh.done, 0);
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, kTmemColumns);
  }
}

std::mutex g_rows_mu;

template <int FMT, int D>
int launch_t(const RowsArgs& a, const OwnArgs& own, cudaStream_t stream) {
  constexpr int kBytes = Smem<FMT, D>::kBytes;
  static uint64_t done_mask = 0;  // guarded by g_rows_mu
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(g_rows_mu);
    if (!(done_mask >> dev & 1)) {
      if (cudaFuncSetAttribute(rows_kernel<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) != cudaSuccess)
        return KVQ_ERR_CUDA;
      done_mask |= 1ull << dev;
    }
  }
  const int64_t blocks =
      (int64_t)a.row_tiles * a.desc.num_kv_heads * a.splits + (own.units + kOwnWarps - 1) / kOwnWarps;
  if (blocks <= 0) return KVQ_OK;
  if (blocks > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  rows_kernel<FMT, D><<<(unsigned)blocks, kThreads, kBytes, stream>>>(a, own);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace

// One CTA per SM: units are cut along their positions until they fill the device, in pieces of
// at least two tiles (one per stream when the rows fit one row tile).  Groups of unequal
// lengths may be cut into up to four times the splits that equal ones would need; the device
// chooses among them (find_unit).
RowsPlan plan_rows(int num_kv_heads, int group, int n_tokens, int num_groups, int max_len, int ctas) {
  RowsPlan p;
  const int64_t rows = (int64_t)n_tokens * group;
  p.row_tiles = num_groups > 32 ? (int)(rows / kRowTile + num_groups)  // find_unit's slots
                                : (int)((rows + (int64_t)num_groups * (kRowTile - 1)) / kRowTile);
  const int64_t units = std::max<int64_t>(1, (int64_t)p.row_tiles * num_kv_heads);
  int64_t want = std::max<int64_t>(1, ctas / units);
  if (num_groups > 1 && num_groups <= 32 && want > 1) want = std::min<int64_t>(4 * want, std::max(1, ctas / num_kv_heads));
  const int64_t len = std::max(max_len, 1);
  int64_t chunk = (len + want - 1) / want;
  chunk = std::max<int64_t>((chunk + kKvTile - 1) / kKvTile * kKvTile, 2 * kKvTile);
  p.min_chunk = (int)std::min<int64_t>(chunk, 0x7fffff00);
  p.splits = (int)((len + chunk - 1) / chunk);
  p.ctas = ctas;
  return p;
}

// A warp per split, as many splits as the device holds warps of own units, whole blocks; no
// split is longer than a sequence (with more pairs than slots the even share is).
int plan_own(int num_kv_heads, int batch, int max_seq_len, int* ctas) {
  const int64_t pairs = (int64_t)std::max(batch, 1) * num_kv_heads;
  const int64_t slots = (int64_t)kTargetCtas * kOwnWarps;
  const int64_t l = std::min<int64_t>((pairs * max_seq_len + slots - 1) / slots, max_seq_len);
  const int split = (int)std::max<int64_t>((l + kTile - 1) / kTile * kTile, kTile);
  const int64_t units = pairs * ((max_seq_len + split - 1) / split);
  *ctas = (int)std::min<int64_t>((units + kOwnWarps - 1) / kOwnWarps, 0x7fffffff);
  return split;
}

size_t rows_partial_bytes(int n_tokens, int num_q_heads, int head_dim, int splits) {
  const size_t n = (size_t)n_tokens * num_q_heads * splits;
  return n * ((size_t)head_dim + 2) * sizeof(float);
}

int launch_rows(const RowsArgs& a, const OwnArgs& own, cudaStream_t stream) {
  const int f = a.desc.fmt, d = a.desc.head_dim;
  if (f == KVQ_FMT_Q8_0 && d == 128) return launch_t<KVQ_FMT_Q8_0, 128>(a, own, stream);
  if (f == KVQ_FMT_Q8_0 && d == 64) return launch_t<KVQ_FMT_Q8_0, 64>(a, own, stream);
  if (f == KVQ_FMT_Q4_0 && d == 128) return launch_t<KVQ_FMT_Q4_0, 128>(a, own, stream);
  if (f == KVQ_FMT_Q4_0 && d == 64) return launch_t<KVQ_FMT_Q4_0, 64>(a, own, stream);
  if (f == KVQ_FMT_LUT4 && d == 128) return launch_t<KVQ_FMT_LUT4, 128>(a, own, stream);
  if (f == KVQ_FMT_LUT4 && d == 64) return launch_t<KVQ_FMT_LUT4, 64>(a, own, stream);
  if (f == KVQ_FMT_NVFP4 && d == 128) return launch_t<KVQ_FMT_NVFP4, 128>(a, own, stream);
  if (f == KVQ_FMT_NVFP4 && d == 64) return launch_t<KVQ_FMT_NVFP4, 64>(a, own, stream);
  return KVQ_ERR_UNSUPPORTED;
}

}  // namespace kvq
