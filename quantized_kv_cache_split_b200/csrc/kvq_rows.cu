// Attention of many query rows over the quantized cache (sm_100a): prompt attention (the
// new tokens of each request over its own positions) and the shared part of prefix decode
// (the tokens of every request of a group over the group's prefix).
//
//   S = Q K^T,  P = 2^(S sm_scale log2(e) - m),  O = P V,  l = sum P
//
// with the running maximum m of a streaming softmax, one pass over the positions.  Both
// products run on the fifth-generation tensor cores.  One CTA (17 warps) per unit:
// (group, KV head, 256 query rows, split of the positions).
//
//   warps 0-3, 4-7   softmax of row tile 0 / 1 (stream 0 / 1): one thread per row.  Scores
//                    come from TMEM, weights go back to TMEM as fp16 (the A operand of P V)
//                    over the scores.  The accumulator is rescaled only when the maximum
//                    has grown by more than 2^8: until then the weights stay below 2^15.
//   warps 8-15       dequantize: codes and scales of a 128-position K or V tile from global
//                    memory to registers, one tile ahead, then as fp16 to shared memory.
//   warp 16          issues the MMAs.
//
// A unit of more than 128 rows runs its two row tiles against the same K / V tiles, so a
// tile is dequantized once for 256 rows.  A unit of at most 128 rows gives both streams
// the same rows and every other tile each; the streams' results are merged at the end.
//
// Roundings: K and V values to fp16 (2^-11 relative, as code * scale; nvfp4 first its block
// scale times vector scale), the lut4 query after its rotation to fp16, the weights to fp16 with 7 bits of headroom.  Scores, maxima, sums
// and accumulators are fp32.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "kvq_decode_common.cuh"
#include "kvq_rows.h"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kSoftmaxWarps = 8, kFillWarps = 8;
constexpr int kMmaWarp = kSoftmaxWarps + kFillWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kFillThreads = 32 * kFillWarps;
constexpr float kWeightBits = 7.f;   // weights are 2^(s - m + 7)
constexpr float kRescaleBits = 8.f;  // growth of the maximum before the accumulator is rescaled
constexpr uint32_t kTmemColumns = 512;
// q8_0 and nvfp4 values enter the products halved (their rounded code * scale can pass the
// largest fp16 value by a step); the factor goes into the score scale and the output.
template <int FMT>
constexpr float kUnhalve = FMT == KVQ_FMT_Q8_0 || FMT == KVQ_FMT_NVFP4 ? 2.f : 1.f;

struct Shared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];  // K / V tile slots
  uint64_t s_full[2], p_full[2];                          // scores / weights of a stream
  uint64_t done;                                          // every MMA completed
  uint32_t tmem;
  int unit[6];  // group, first token row, rows, positions, new tokens, valid
  float merge_m[128], merge_l[128];
};

template <int D>
struct Smem {
  static constexpr int kTileBytes = 128 * D * 2;  // 128 rows of D fp16
  static constexpr int kQ = 0;                    // two row tiles
  static constexpr int kK = 2 * kTileBytes;       // two slots
  static constexpr int kV = 4 * kTileBytes;       // two slots
  static constexpr int kBars = 6 * kTileBytes;
  static constexpr int kBytes = kBars + (int)sizeof(Shared) + 1024;  // slack: 1024-byte alignment
};

// Byte offset of 16-byte chunk c of a row in a [128][D] fp16 tile: column groups of 64, 128-byte
// swizzle.
__device__ __forceinline__ uint32_t tile_offset(int row, int c) {
  return (uint32_t)((c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

// ------------------------------------------------------------------ dequantization
template <int FMT, int D>
struct Fill {
  using C = Cfg<FMT, D>;
  static constexpr int kChunks = C::CROW / 16;               // 16-byte code chunks of a row
  static constexpr int kTasks = 128 * kChunks / kFillThreads;  // chunks per thread and tile
  static_assert(kTasks >= 1, "a chunk for every thread");
  uint4 code[kTasks];
  uint32_t scale[kTasks];  // fp16 scale, or nvfp4: two E4M3 bytes
  float vec[C::kNv ? kTasks : 1];
};

template <int FMT, int D>
__device__ __forceinline__ uint4 dequant8(uint32_t w0, uint32_t w1, __half2 d, const Lut& lut) {
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
    r = make_uint4(hmul2u(prmt(L0, H0, 0x5140u), d), hmul2u(prmt(L0, H0, 0x7362u), d),
                   hmul2u(prmt(L1, H1, 0x5140u), d), hmul2u(prmt(L1, H1, 0x7362u), d));
  }
  return r;
}

// This thread's codes and scales of a tile; rows at or past n_valid are zero.  base0 / base1:
// cache rows of the tile's two 64-position halves (negative: nothing to read).
template <int FMT, int D>
__device__ __forceinline__ void fill_load(Fill<FMT, D>& f, const uint8_t* __restrict__ codes,
                                          const uint8_t* __restrict__ scales, int64_t base0, int64_t base1,
                                          int n_valid, int tid) {
  using C = Cfg<FMT, D>;
  using F = Fill<FMT, D>;
#pragma unroll
  for (int i = 0; i < F::kTasks; ++i) {
    const int task = i * kFillThreads + tid;
    const int row = task / F::kChunks, j = task % F::kChunks;
    const int64_t base = row < 64 ? base0 : base1;
    f.code[i] = make_uint4(0u, 0u, 0u, 0u);
    f.scale[i] = 0u;
    if constexpr (C::kNv) f.vec[i] = 0.f;
    if (row < n_valid && base >= 0) {
      const int64_t at = base + (row & 63);
      f.code[i] = __ldg(reinterpret_cast<const uint4*>(codes + at * C::CROW) + j);
      const uint8_t* s = scales + at * C::SROW;
      if constexpr (C::kQ8) {
        f.scale[i] = __ldg(reinterpret_cast<const uint16_t*>(s) + (j >> 1));
      } else if constexpr (C::kQ4) {
        f.scale[i] = __ldg(reinterpret_cast<const uint16_t*>(s) + j);
      } else if constexpr (C::kLut) {
        f.scale[i] = __ldg(reinterpret_cast<const uint16_t*>(s));
      } else {
        f.scale[i] = __ldg(reinterpret_cast<const uint16_t*>(s) + j);
        f.vec[i] = __ldg(reinterpret_cast<const float*>(s + D / 16));
      }
    }
  }
}

template <int FMT, int D>
__device__ __forceinline__ void fill_store(const Fill<FMT, D>& f, uint8_t* tile, int tid, const Lut& lut) {
  using C = Cfg<FMT, D>;
  using F = Fill<FMT, D>;
#pragma unroll
  for (int i = 0; i < F::kTasks; ++i) {
    const int task = i * kFillThreads + tid;
    const int row = task / F::kChunks, j = task % F::kChunks;
    const uint32_t w[4] = {f.code[i].x, f.code[i].y, f.code[i].z, f.code[i].w};
    // The threads of a row that write the second column group take their chunks in another
    // order, so that eight neighbours write eight different bank groups.
    if constexpr (C::kQ8) {
      const __half2 d = __half2half2(__ushort_as_half((unsigned short)f.scale[i]));
      const bool flip = (j >> 2) & 1;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 v = dequant8<FMT, D>(flip ? w[2 - 2 * c] : w[2 * c], flip ? w[3 - 2 * c] : w[2 * c + 1], d, lut);
        *reinterpret_cast<uint4*>(tile + tile_offset(row, 2 * j + (c ^ (int)flip))) = v;
      }
    } else {
      const bool flip = (j >> 1) & 1;
      __half2 d0, d1;
      if constexpr (C::kNv) {
        d0 = __float2half2_rn(e4m3_float(f.scale[i] & 0xffu) * f.vec[i]);
        d1 = __float2half2_rn(e4m3_float(f.scale[i] >> 8) * f.vec[i]);
      } else {
        d0 = d1 = __half2half2(__ushort_as_half((unsigned short)f.scale[i]));
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool second = flip ? (c < 2) : (c >= 2);  // chunk c ^ 2 flip is in the second half
        const uint4 v = dequant8<FMT, D>(flip ? w[c ^ 2] : w[c], 0u, second ? d1 : d0, lut);
        *reinterpret_cast<uint4*>(tile + tile_offset(row, 4 * j + (flip ? c ^ 2 : c))) = v;
      }
    }
  }
}

// ------------------------------------------------------------------ unit lookup
// Row tile `t` (over all groups): its group and first row.  One warp; the lanes take
// consecutive ranges of groups.
__device__ __forceinline__ void find_unit(const RowsArgs& a, int t, int lane, int* unit) {
  const int per = (a.num_groups + 31) / 32;
  const int g0 = min(lane * per, a.num_groups), g1 = min(g0 + per, a.num_groups);
  auto tokens = [&](int g, int& first) {
    if (!a.offsets) {
      first = 0;
      return a.n_tokens;
    }
    first = a.offsets[g];
    const int end = a.offsets[g + 1];
    if (first < 0 || end < first || end > a.n_tokens) {
      set_flag(a.flags, KVQ_FLAG_BAD_SEQLEN);
      return 0;
    }
    return end - first;
  };
  int mine = 0, first;
  for (int g = g0; g < g1; ++g) mine += (tokens(g, first) * a.group + kRowTile - 1) / kRowTile;
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  before -= mine;
  if (lane == 0) unit[5] = 0;
  __syncwarp();
  if (t >= before && t < before + mine) {
    int k = t - before;
    for (int g = g0; g < g1; ++g) {
      const int n = tokens(g, first);
      const int tiles = (n * a.group + kRowTile - 1) / kRowTile;
      if (k < tiles) {
        // the last rows of a causal group see the most positions: they start first
        const int tile = a.causal ? tiles - 1 - k : k;
        int len = a.lens[g];
        if (len < 0 || len > a.max_len || len > (int64_t)a.max_pages * a.desc.page_size) {
          set_flag(a.flags, KVQ_FLAG_BAD_SEQLEN);
          len = 0;
        }
        unit[0] = g;
        unit[1] = tile * kRowTile;
        unit[2] = min(n * a.group - tile * kRowTile, kRowTile);
        unit[3] = len;
        unit[4] = first;
        unit[5] = n;
        break;
      }
      k -= tiles;
    }
  }
  __syncwarp();
}

// ------------------------------------------------------------------ the kernel
template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const RowsArgs a) {
  using C = Cfg<FMT, D>;
  using S = Smem<D>;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  Shared& sh = *reinterpret_cast<Shared*>(smem + S::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hkv = a.desc.num_kv_heads, G = a.group;
  // block: split fastest, then KV head, then row tile
  const int split = blockIdx.x % a.splits;
  const int kvh = blockIdx.x / a.splits % hkv;
  const int rt = blockIdx.x / a.splits / hkv;

  if (warp == 0) find_unit(a, rt, lane, sh.unit);
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem, kTmemColumns);
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        bar_init(&sh.k_full[i], kFillWarps);
        bar_init(&sh.v_full[i], kFillWarps);
        bar_init(&sh.k_empty[i], 1);
        bar_init(&sh.v_empty[i], 1);
        bar_init(&sh.s_full[i], 1);
        bar_init(&sh.p_full[i], kSoftmaxWarps / 2);
      }
      bar_init(&sh.done, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  }
  __syncthreads();
  const int g = sh.unit[0], row0 = sh.unit[1], rows = sh.unit[2], len = sh.unit[3], tok0 = sh.unit[4], n = sh.unit[5];
  // positions of this split that any row of the unit sees
  const int last = n > 0 ? row_limit(len, n, (row0 + rows - 1) / G, a.causal) : 0;
  const int begin = split * a.chunk;
  const int end = min(min(last, len), begin + a.chunk);
  const int tiles = end > begin ? (end - begin + kKvTile - 1) / kKvTile : 0;
  const bool shared_tiles = rows > 128;  // both streams take every tile; else every other one
  const bool live = n > 0 && (tiles > 0 || a.out != nullptr);

  // query rows, fp16, K-major, 128-byte swizzle; rows past the unit's are zero
  if (live && tiles > 0) {
    const __half* q = static_cast<const __half*>(a.q);
    const bool zero = a.sm_scale == 0.f;
    const uint32_t flip = a.sm_scale < 0.f ? 0x80008000u : 0u;  // the scale's sign goes into the query
    if constexpr (!C::kLut) {
      constexpr int kC = D / 8;
      for (int i = tid; i < kRowTile * kC; i += kThreads) {
        const int r = i / kC, c = i % kC;
        const int rr = shared_tiles ? r : r & 127;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (rr < rows && !zero) {
          const int t = (row0 + rr) / G, h = (row0 + rr) % G;
          v = __ldg(reinterpret_cast<const uint4*>(q + ((int64_t)(tok0 + t) * a.num_q_heads + kvh * G + h) * D) + c);
          v.x ^= flip; v.y ^= flip; v.z ^= flip; v.w ^= flip;
        }
        *reinterpret_cast<uint4*>(smem + S::kQ + (r >> 7) * S::kTileBytes + tile_offset(r & 127, c)) = v;
      }
    } else {
      // rotated: (1/sqrt(D)) H (signs .* q); a warp per row, lane l holds E consecutive elements
      constexpr int E = D / 32;
      for (int r = warp; r < kRowTile; r += kThreads / 32) {
        const int rr = shared_tiles ? r : r & 127;
        float y[E];
#pragma unroll
        for (int k = 0; k < E; ++k) y[k] = 0.f;
        if (rr < rows && !zero) {
          const int t = (row0 + rr) / G, h = (row0 + rr) % G;
          const __half* src = q + ((int64_t)(tok0 + t) * a.num_q_heads + kvh * G + h) * D + lane * E;
#pragma unroll
          for (int k = 0; k < E; ++k) y[k] = __half2float(src[k]) * (float)a.desc.signs[lane * E + k];
        }
#pragma unroll
        for (int h = 1; h < E; h <<= 1)
#pragma unroll
          for (int k = 0; k < E; ++k)
            if (!(k & h)) {
              const float u = y[k], v = y[k + h];
              y[k] = u + v;
              y[k + h] = u - v;
            }
#pragma unroll
        for (int b = 1; b < 32; b <<= 1)
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const float o = __shfl_xor_sync(0xffffffffu, y[k], b);
            y[k] = (lane & b) ? o - y[k] : y[k] + o;
          }
        const float cs = D == 64 ? 0.125f : 0.08838834764831845f;  // 1/sqrt(D)
        uint8_t* dst = smem + S::kQ + (r >> 7) * S::kTileBytes + tile_offset(r & 127, lane * E / 8) + (lane * E % 8) * 2;
#pragma unroll
        for (int k = 0; k < E; k += 2)
          *reinterpret_cast<uint32_t*>(dst + 2 * k) = pack_h2(y[k] * cs, y[k + 1] * cs) ^ flip;
      }
    }
    fence_async_shared();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  bool ok = true;

  if (live && tiles > 0) {
    if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA
      if (lane == 0) {
        constexpr uint32_t kIdS = mma_idesc(128, kKvTile, false);
        constexpr uint32_t kIdO = mma_idesc(128, D, true);
        auto qk = [&](int s, int slot) {
          const uint32_t qa = smem_u32(smem + S::kQ + s * S::kTileBytes);
          const uint32_t ka = smem_u32(smem + S::kK + slot * S::kTileBytes);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
            mma_ss(tmem + s * 128, mma_desc(qa + off, 16, 1024), mma_desc(ka + off, 16, 1024), kIdS, k > 0);
          }
          mma_commit(&sh.s_full[s]);
        };
        auto pv = [&](int s, int slot, bool first) {
          const uint32_t va = smem_u32(smem + S::kV + slot * S::kTileBytes);
#pragma unroll
          for (int k = 0; k < kKvTile / 16; ++k)
            mma_ts(tmem + 256 + s * D, tmem + s * 128 + k * 8, mma_desc(va + k * 2048, 16384, 1024), kIdO,
                   !first || k > 0);
        };
        if (shared_tiles) {
          ok = bar_wait(&sh.k_full[0], 0);
          if (ok) {
            tc_fence_after();
            qk(0, 0);
            qk(1, 0);
            mma_commit(&sh.k_empty[0]);
          }
          for (int t = 0; ok && t < tiles; ++t) {
            const int slot = t & 1, next = (t + 1) & 1;
            ok = bar_wait(&sh.v_full[slot], t >> 1 & 1);
            for (int s = 0; ok && s < 2; ++s) {
              ok = bar_wait(&sh.p_full[s], t & 1);
              if (!ok) break;
              tc_fence_after();
              pv(s, slot, t == 0);
              if (s == 1) mma_commit(&sh.v_empty[slot]);
              if (t + 1 < tiles) {
                if (s == 0) {
                  ok = bar_wait(&sh.k_full[next], (t + 1) >> 1 & 1);
                  if (!ok) break;
                  tc_fence_after();
                }
                qk(s, next);
                if (s == 1) mma_commit(&sh.k_empty[next]);
              }
            }
          }
        } else {
          for (int s = 0; ok && s < 2 && s < tiles; ++s) {
            ok = bar_wait(&sh.k_full[s], 0);
            if (!ok) break;
            tc_fence_after();
            qk(s, s);
            mma_commit(&sh.k_empty[s]);
          }
          for (int t = 0; ok && t < tiles; ++t) {
            const int s = t & 1, i = t >> 1;
            ok = bar_wait(&sh.v_full[s], i & 1) && bar_wait(&sh.p_full[s], i & 1);
            if (!ok) break;
            tc_fence_after();
            pv(s, s, i == 0);
            mma_commit(&sh.v_empty[s]);
            if (t + 2 < tiles) {
              ok = bar_wait(&sh.k_full[s], (i + 1) & 1);
              if (!ok) break;
              tc_fence_after();
              qk(s, s);
              mma_commit(&sh.k_empty[s]);
            }
          }
        }
        mma_commit(&sh.done);
      }
      __syncwarp();
    } else if (warp >= kSoftmaxWarps) {
      // ---------------------------------------------------------------- dequantize
      // K0 K1 V0 K2 V1 K3 ...: the order in which the MMAs of either mode need the tiles
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
      const uint8_t* kc = static_cast<const uint8_t*>(a.k_codes);
      const uint8_t* ks = static_cast<const uint8_t*>(a.k_scales);
      const uint8_t* vc = static_cast<const uint8_t*>(a.v_codes);
      const uint8_t* vs = static_cast<const uint8_t*>(a.v_scales);
      const int ps = a.desc.page_size;
      // cache row of position p (a multiple of 64) of this unit's KV head; -1: none
      auto base_of = [&](int p) -> int64_t {
        if (p >= end) return -1;
        const int pg = p / ps;
        const int page = a.table ? __ldg(a.table + (int64_t)g * a.max_pages + pg) : g * a.max_pages + pg;
        if (page < 0 || page >= a.desc.num_pages) {
          set_flag(a.flags, KVQ_FLAG_BAD_PAGE);
          return -1;
        }
        return ((int64_t)page * hkv + kvh) * ps + (p - pg * ps);
      };
      Fill<FMT, D> fk, fv;
      auto load_k = [&](int t) {
        const int p = begin + t * kKvTile;
        fill_load<FMT, D>(fk, kc, ks, base_of(p), base_of(p + 64), end - p, ft);
      };
      auto load_v = [&](int t) {
        const int p = begin + t * kKvTile;
        fill_load<FMT, D>(fv, vc, vs, base_of(p), base_of(p + 64), end - p, ft);
      };
      auto put_k = [&](int t) {
        ok = t < 2 || bar_wait(&sh.k_empty[t & 1], (t >> 1 & 1) ^ 1);
        if (!ok) return;
        fill_store<FMT, D>(fk, smem + S::kK + (t & 1) * S::kTileBytes, ft, lut);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.k_full[t & 1]);
      };
      auto put_v = [&](int t) {
        ok = t < 2 || bar_wait(&sh.v_empty[t & 1], (t >> 1 & 1) ^ 1);
        if (!ok) return;
        fill_store<FMT, D>(fv, smem + S::kV + (t & 1) * S::kTileBytes, ft, lut);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.v_full[t & 1]);
      };
      load_k(0);
      load_v(0);
      put_k(0);
      if (tiles > 1) {
        load_k(1);
        put_k(1);
      }
      if (tiles > 2) load_k(2);
      for (int t = 0; ok && t < tiles; ++t) {
        put_v(t);
        if (t + 1 < tiles) load_v(t + 1);
        if (ok && t + 2 < tiles) {
          put_k(t + 2);
          if (t + 3 < tiles) load_k(t + 3);
        }
      }
    } else {
      // ---------------------------------------------------------------- softmax
      const int s = warp >> 2;
      const int r = tid & 127;  // row of the row tile = TMEM lane
      const int rr = shared_tiles ? s * 128 + r : r;
      const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's lanes
      const float scale = (a.sm_scale == 0.f ? 1.f : fabsf(a.sm_scale)) * kLog2e * kUnhalve<FMT>;
      const int limit = rr < rows ? min(row_limit(len, n, (row0 + rr) / G, a.causal), end) : end;
      const int steps = shared_tiles ? tiles : (tiles - s + 1) / 2;
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < steps; ++i) {
        const int t = shared_tiles ? i : 2 * i + s;
        const int lim = limit - begin - t * kKvTile;  // visible columns of this row in the tile
        ok = bar_wait(&sh.s_full[s], i & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ts = at + s * 128;
        const bool mask = __any_sync(0xffffffffu, lim < kKvTile);
        // maximum
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int c = 0; c < kKvTile; c += 32) {
          float v[32];
          tmem_ld32(ts + c, v);
          tmem_wait_ld32(v);
          if (mask) {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = c + k < lim ? v[k] : -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) mx[k & 3] = fmaxf(mx[k & 3], v[k]);
        }
        const float tm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
        const bool grow = tm > m + kRescaleBits || (m == -INFINITY && tm > -INFINITY);
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(m - tm) : 1.f;  // m = -inf: 0
          if (grow) m = tm;
          l *= f;
          // the scores of this tile were issued after the last P V of this stream, so the
          // accumulator is at rest
          if (i > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float v[32];
              tmem_ld32(at + 256 + s * D + c, v);
              tmem_wait_ld32(v);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] *= f;
              tmem_st32(at + 256 + s * D + c, reinterpret_cast<const uint32_t*>(v));
            }
            tmem_wait_st();
          }
        }
        const float off = m == -INFINITY ? 0.f : kWeightBits - m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c = 0; c < kKvTile; c += 64) {
          float v[64];
          uint32_t p[32];
          tmem_ld32(ts + c, v);
          tmem_ld32(ts + c + 32, v + 32);
          tmem_wait_ld32(v);
          tmem_wait_ld32(v + 32);
          if (mask) {
#pragma unroll
            for (int k = 0; k < 64; ++k) v[k] = c + k < lim ? v[k] : -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            const float e0 = ex2(fmaf(v[k], scale, off)), e1 = ex2(fmaf(v[k + 1], scale, off));
            sum[(k >> 1) & 3] += e0 + e1;
            p[k >> 1] = pack_h2(e0, e1);
          }
          tmem_st32(ts + c / 2, p);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.p_full[s]);
      }
      if (ok) ok = bar_wait(&sh.done, 0);
      tc_fence_after();
      // ---------------------------------------------------------------- results
      m -= kWeightBits;  // the weights were 2^(s - m + 7)
      const float vscale = kUnhalve<FMT>;
      float f0 = vscale, f1 = 0.f;
      float4* stage = reinterpret_cast<float4*>(smem + S::kK);  // [D / 4][128], stream 1's rows
      if (!shared_tiles) {
        // streams 0 and 1 hold the same rows: stream 1 hands its sums to stream 0
        if (s == 1) {
          sh.merge_m[r] = m;
          sh.merge_l[r] = l;
          if (steps > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float v[32];
              tmem_ld32(at + 256 + s * D + c, v);
              tmem_wait_ld32(v);
#pragma unroll
              for (int k = 0; k < 32; k += 4)
                stage[(c + k) / 4 * 128 + r] = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
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
        const bool write = ok && rr < rows;
        const int64_t row = write ? (int64_t)(tok0 + (row0 + rr) / G) * a.num_q_heads + kvh * G + (row0 + rr) % G : 0;
        const int64_t part = row * a.splits + split;
        if (a.out) {
          const float inv = l > 0.f ? 1.f / l : 0.f;
          f0 *= inv;
          f1 *= inv;
        } else if (write) {
          a.part_m[part] = m;
          a.part_l[part] = l;
        }
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(at + 256 + s * D + c, v);
          tmem_wait_ld32(v);
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float4 o = make_float4(v[k] * f0, v[k + 1] * f0, v[k + 2] * f0, v[k + 3] * f0);
            if (f1 != 0.f) {
              const float4 x = stage[(c + k) / 4 * 128 + r];
              o.x = fmaf(x.x, f1, o.x); o.y = fmaf(x.y, f1, o.y);
              o.z = fmaf(x.z, f1, o.z); o.w = fmaf(x.w, f1, o.w);
            }
            v[k] = o.x; v[k + 1] = o.y; v[k + 2] = o.z; v[k + 3] = o.w;
          }
          if (write) {
            if (!a.out || !a.out_f16) {
              float* dst = (a.out ? static_cast<float*>(a.out) + row * D : a.part_o + part * D) + c;
#pragma unroll
              for (int k = 0; k < 32; k += 4)
                *reinterpret_cast<float4*>(dst + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            } else {
              __half* dst = static_cast<__half*>(a.out) + row * D + c;
#pragma unroll
              for (int k = 0; k < 32; k += 8)
                *reinterpret_cast<uint4*>(dst + k) = make_uint4(pack_h2(v[k], v[k + 1]), pack_h2(v[k + 2], v[k + 3]),
                                                                pack_h2(v[k + 4], v[k + 5]), pack_h2(v[k + 6], v[k + 7]));
            }
          }
        }
      }
    }
  } else if (live && warp < kSoftmaxWarps && tid < rows) {
    // no position at all: the rows are zero
    const int64_t row = (int64_t)(tok0 + (row0 + tid) / G) * a.num_q_heads + kvh * G + (row0 + tid) % G;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + row * D * (a.out_f16 ? 2 : 4));
    for (int k = 0; k < D * (a.out_f16 ? 2 : 4) / 16; ++k) dst[k] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (!ok) set_flag(a.flags, KVQ_FLAG_TIMEOUT);
  // the MMAs still in flight (after a wait that gave up) end before the TMEM is freed
  if (warp == kMmaWarp && lane == 0 && live && tiles > 0) (void)bar_wait(&sh.done, 0);
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, kTmemColumns);
  }
}

std::mutex g_rows_mu;

template <int FMT, int D>
int launch_t(const RowsArgs& a, cudaStream_t stream) {
  constexpr int kBytes = Smem<D>::kBytes;
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
  const int64_t blocks = (int64_t)a.row_tiles * a.desc.num_kv_heads * a.splits;
  if (blocks <= 0) return KVQ_OK;
  if (blocks > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  rows_kernel<FMT, D><<<(unsigned)blocks, kThreads, kBytes, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace

// One CTA per SM: a unit is cut along its positions until the units fill the device, in
// pieces of at least two tiles (one per stream when the rows fit one row tile).
RowsPlan plan_rows(int num_kv_heads, int group, int n_tokens, int num_groups, int max_len) {
  RowsPlan p;
  const int64_t rows = (int64_t)n_tokens * group;
  p.row_tiles = (int)((rows + (int64_t)num_groups * (kRowTile - 1)) / kRowTile);
  const int64_t units = std::max<int64_t>(1, (int64_t)p.row_tiles * num_kv_heads);
  const int64_t want = std::max<int64_t>(1, kTargetCtas / units);
  const int64_t len = std::max(max_len, 1);
  int64_t chunk = (len + want - 1) / want;
  chunk = std::max<int64_t>((chunk + kKvTile - 1) / kKvTile * kKvTile, 2 * kKvTile);
  p.chunk = (int)std::min<int64_t>(chunk, 0x7fffff00);
  p.splits = (int)((len + chunk - 1) / chunk);
  return p;
}

size_t rows_partial_bytes(int n_tokens, int num_q_heads, int head_dim, int splits) {
  const size_t n = (size_t)n_tokens * num_q_heads * splits;
  return n * ((size_t)head_dim + 2) * sizeof(float);
}

int launch_rows(const RowsArgs& a, cudaStream_t stream) {
  const int f = a.desc.fmt, d = a.desc.head_dim;
  if (f == KVQ_FMT_Q8_0 && d == 128) return launch_t<KVQ_FMT_Q8_0, 128>(a, stream);
  if (f == KVQ_FMT_Q8_0 && d == 64) return launch_t<KVQ_FMT_Q8_0, 64>(a, stream);
  if (f == KVQ_FMT_Q4_0 && d == 128) return launch_t<KVQ_FMT_Q4_0, 128>(a, stream);
  if (f == KVQ_FMT_Q4_0 && d == 64) return launch_t<KVQ_FMT_Q4_0, 64>(a, stream);
  if (f == KVQ_FMT_LUT4 && d == 128) return launch_t<KVQ_FMT_LUT4, 128>(a, stream);
  if (f == KVQ_FMT_LUT4 && d == 64) return launch_t<KVQ_FMT_LUT4, 64>(a, stream);
  if (f == KVQ_FMT_NVFP4 && d == 128) return launch_t<KVQ_FMT_NVFP4, 128>(a, stream);
  if (f == KVQ_FMT_NVFP4 && d == 64) return launch_t<KVQ_FMT_NVFP4, 64>(a, stream);
  return KVQ_ERR_UNSUPPORTED;
}

}  // namespace kvq
