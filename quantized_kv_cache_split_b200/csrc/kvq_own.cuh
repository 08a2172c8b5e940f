// Decode attention of one token over its own positions, one warp per split: the requests' part
// of prefix decode.  The sequences are short and many, so the unit is a warp that streams
// through its split by itself (blocks of 64 positions, K and V staged in its own slice of
// shared memory, the next K block in flight during the V pass), without a barrier: latency is
// hidden by the other warps of the SM.
//
//   S = K Q^T (mma.sync m16n8k16: 16 positions x 8 heads), streaming softmax per head,
//   O^T += V^T P (dims x heads); V enters as fp16 code * scale, P as fp16.
#pragma once

#include "kvq_decode_common.cuh"
#include "kvq_rows.h"

namespace kvq {
namespace {

constexpr float kOwnWeightBits = 7.f;  // weights are 2^(s - m + 7): above fp16's smallest steps

template <int FMT, int D>
struct Own {
  using C = Cfg<FMT, D>;
  static constexpr int kCodes = kTile * C::CROW, kScales = kTile * C::SROW;
  static constexpr int kBytes = 2 * (kCodes + kScales);  // a K and a V block
  static constexpr float kUnhalve = C::kQ8 || C::kNv ? 2.f : 1.f;
};

// Copy a block (64 positions of a page) into the warp's slice, 16-byte chunks swizzled as the
// fragment loads expect.
template <int FMT, int D>
__device__ __forceinline__ void own_stage(uint8_t* dst, const uint8_t* __restrict__ codes,
                                          const uint8_t* __restrict__ scales, int row, int lane) {
  using C = Cfg<FMT, D>;
  using O = Own<FMT, D>;
  constexpr int kChunks = C::CROW / 16;
  const uint8_t* src = codes + (int64_t)row * C::CROW;
#pragma unroll
  for (int i = 0; i < O::kCodes / 16 / 32; ++i) {
    const int k = i * 32 + lane, r = k / kChunks, c = k % kChunks;
    cp_async16(dst + r * C::CROW + ((c ^ swz<FMT, D>(r)) << 4), src + k * 16);
  }
  const uint8_t* ss = scales + (int64_t)row * C::SROW;
  for (int k = lane; k < O::kScales / 16; k += 32) cp_async16(dst + O::kCodes + k * 16, ss + k * 16);
}

// acc += V^T P for the 16 rows s0 .. s0 + 15 of a staged block (those at or past n_valid as
// zeros); p01, p89: the weights' B fragments.
template <int FMT, int D>
__device__ __forceinline__ void own_v(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int s0,
                                      int n_valid, uint32_t p01, uint32_t p89, int lane, const Lut& lut,
                                      float (&acc)[D / 16][4]) {
  using C = Cfg<FMT, D>;
  const int r = lane >> 2, c = lane & 3;
  if constexpr (C::kMag) {
    constexpr int NW = C::NBLK / 2;
    uint32_t ws[4][NW];  // scale words of rows s0 + {2c, 2c + 1, 2c + 8, 2c + 9}
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int slot = s0 + 2 * c + (q & 1) + 8 * (q >> 1);
#pragma unroll
      for (int w = 0; w < NW; ++w) ws[q][w] = slot < n_valid ? lds32(scales + slot * C::SROW + 4 * w) : 0u;
    }
    const int mi = lane >> 3, row = s0 + 8 * (mi & 1) + (lane & 7);
    const uint8_t* rp = codes + row * C::CROW;
    const int sw = swz<FMT, D>(row);
#pragma unroll
    for (int cb = 0; cb < C::CROW / 16; cb += 2) {
      uint32_t R[2][2];  // chunk cb + j, rows 2c, 2c + 1 (+ 8 h)
      ldsm_x4_trans(rp + (((cb + (mi >> 1)) ^ sw) << 4), R[0][0], R[0][1], R[1][0], R[1][1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int ch = cb + j, blk = C::kQ4 ? ch : ch >> 1;
        const uint32_t sel = (blk & 1) ? 0x7632u : 0x5410u;
        const __half2 d0 = u32_as_h2(prmt(ws[0][blk >> 1], ws[1][blk >> 1], sel));
        const __half2 d1 = u32_as_h2(prmt(ws[2][blk >> 1], ws[3][blk >> 1], sel));
        if constexpr (C::kQ4) {
          auto val = [](uint32_t x, uint32_t mask, uint32_t magic, uint32_t neg, __half2 d) {
            return h2_as_u32(__hmul2(__hadd2(u32_as_h2((x & mask) | magic), u32_as_h2(neg)), d));
          };
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t x0 = R[j][0] >> (8 * k), x1 = R[j][1] >> (8 * k);
            mma16816(acc[2 * ch + k], val(x0, 0x000F000Fu, kMagic, 0xE408E408u, d0),
                     val(x0, 0x00F000F0u, kMagic64, 0xD480D480u, d0), val(x1, 0x000F000Fu, kMagic, 0xE408E408u, d1),
                     val(x1, 0x00F000F0u, kMagic64, 0xD480D480u, d1), p01, p89);
          }
        } else {
          const __half2 half = u32_as_h2(0x38003800u), bias = u32_as_h2(0xE080E080u);  // 0.5, -576
          auto val = [&](uint32_t x, uint32_t sel8, __half2 d) {
            return h2_as_u32(__hmul2(__hfma2(u32_as_h2(prmt(x, 0x64646464u, sel8)), half, bias), d));
          };
          const uint32_t x0 = R[j][0] ^ 0x80808080u, x1 = R[j][1] ^ 0x80808080u;
          mma16816(acc[ch], val(x0, 0x4240u, d0), val(x0, 0x4341u, d0), val(x1, 0x4240u, d1), val(x1, 0x4341u, d1), p01,
                   p89);
        }
      }
    }
  } else {
    auto code = [&](int slot) -> const uint8_t* {
      const int o = C::RAWB * r;
      return codes + slot * C::CROW + (((o >> 4) ^ swz<FMT, D>(slot)) << 4) + (o & 15);
    };
    auto scale = [&](int slot) -> float {
      if (slot >= n_valid) return 0.f;
      const uint8_t* srow = scales + slot * C::SROW;
      if constexpr (C::kNv) return e4m3_float(srow[C::E * r / 16]) * *reinterpret_cast<const float*>(srow + D / 16);
      return __half2float(*reinterpret_cast<const __half*>(srow));
    };
    const int sa = s0 + 2 * c, sc = sa + 8;
    const float fa = scale(sa), fb = scale(sa + 1), fc = scale(sc), fd = scale(sc + 1);
    const __half2 dab = __floats2half2_rn(fa, fb), dcd = __floats2half2_rn(fc, fd);
    uint32_t wa[C::NWORD], wb[C::NWORD], e[2][C::E];
    v_raw<FMT, D>(code(sa), wa);
    v_raw<FMT, D>(code(sa + 1), wb);
    v_dequant_pair<FMT, D>(wa, wb, lut, e[0]);
    v_raw<FMT, D>(code(sc), wa);
    v_raw<FMT, D>(code(sc + 1), wb);
    v_dequant_pair<FMT, D>(wa, wb, lut, e[1]);
    if constexpr (C::kNv) {
      // halved (exact), so that no value passes the fp16 range; what the rounded scale leaves of
      // the exact one is added before the product is rounded
      const __half2 half = u32_as_h2(0x38003800u);
      const float2 ab = __half22float2(dab), cd = __half22float2(dcd);
      const __half2 lab = __floats2half2_rn(fa - ab.x, fb - ab.y), lcd = __floats2half2_rn(fc - cd.x, fd - cd.y);
#pragma unroll
      for (int i = 0; i < C::E; ++i) {
        const __half2 x = __hmul2(u32_as_h2(e[0][i]), half), y = __hmul2(u32_as_h2(e[1][i]), half);
        e[0][i] = h2_as_u32(__hfma2(x, dab, __hmul2(x, lab)));
        e[1][i] = h2_as_u32(__hfma2(y, dcd, __hmul2(y, lcd)));
      }
    } else {
#pragma unroll
      for (int i = 0; i < C::E; ++i) {
        e[0][i] = hmul2u(e[0][i], dab);
        e[1][i] = hmul2u(e[1][i], dcd);
      }
    }
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) mma16816(acc[mt], e[0][2 * mt], e[0][2 * mt + 1], e[1][2 * mt], e[1][2 * mt + 1], p01, p89);
  }
}

// Unit u of the launch: (request, KV head, split), split fastest.  `slice`: this warp's
// Own::kBytes of shared memory, 16-byte aligned.
template <int FMT, int D>
__device__ __forceinline__ void own_unit(const OwnArgs& o, const RowsArgs& a, int64_t u, uint8_t* slice, int lane) {
  using C = Cfg<FMT, D>;
  using O = Own<FMT, D>;
  const int hkv = a.desc.num_kv_heads, G = a.group, ps = a.desc.page_size;
  const int split = (int)(u % o.max_splits);
  const int kvh = (int)(u / o.max_splits % hkv), b = (int)(u / o.max_splits / hkv);
  int len = o.seq_lens[b];
  if (len < 0 || len > o.max_seq_len || len > (int64_t)o.max_pages * ps) {
    if (lane == 0) set_flag(a.flags, KVQ_FLAG_BAD_SEQLEN);
    return;  // (the merge reads no partial of such a request)
  }
  const int begin = split * o.split, end = min(len, begin + o.split);
  if (begin >= end) return;
  const int r = lane >> 2, c = lane & 3;
  const uint8_t* kc = static_cast<const uint8_t*>(a.k_codes);
  const uint8_t* ks = static_cast<const uint8_t*>(a.k_scales);
  const uint8_t* vc = static_cast<const uint8_t*>(a.v_codes);
  const uint8_t* vs = static_cast<const uint8_t*>(a.v_scales);
  auto row_of = [&](int p) -> int {  // first cache row of the block at position p, -1: bad page
    if (p >= end) return 0;
    const int pg = p / ps;
    const int page = o.table ? __ldg(o.table + (int64_t)b * o.max_pages + pg) : b * o.max_pages + pg;
    if (page < 0 || page >= a.desc.num_pages) {
      if (lane == 0) set_flag(a.flags, KVQ_FLAG_BAD_PAGE);
      return -1;
    }
    return (page * hkv + kvh) * ps + (p - pg * ps);
  };
  uint8_t* kt = slice;
  uint8_t* vt = slice + O::kCodes + O::kScales;
  int row = row_of(begin);
  if (row < 0) row = 0;  // any row of the cache: the call is flagged
  own_stage<FMT, D>(kt, kc, ks, row, lane);
  cp_async_commit();
  own_stage<FMT, D>(vt, vc, vs, row, lane);
  cp_async_commit();

  Lut lut;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lut.lo[i] = lut.hi[i] = 0u;
    if constexpr (C::kLut) {
      uint32_t e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = a.desc.codebook[4 * i + k];
      lut.lo[i] = (e[0] & 0xffu) | (e[1] & 0xffu) << 8 | (e[2] & 0xffu) << 16 | (e[3] & 0xffu) << 24;
      lut.hi[i] = e[0] >> 8 | (e[1] >> 8) << 8 | (e[2] >> 8) << 16 | (e[3] >> 8) << 24;
    } else if constexpr (C::kNv) {
      lut.hi[i] = i == 0 ? 0x3E3C3800u : i == 1 ? 0x46444240u : i == 2 ? 0xBEBCB880u : 0xC6C4C2C0u;
    }
  }
  const __half* qh = static_cast<const __half*>(a.q) + ((int64_t)b * a.num_q_heads + kvh * G) * D;
  uint32_t qf[D / 16][2], ql[D / 16][2];
  float corr[D / 32][2];
  {
    QRaw<D> q;
    load_query<FMT, D>(r < G ? qh + r * D : nullptr, a.desc.signs, c, q);
    build_query<FMT, D>(q, c, qf, ql, corr);
  }
  const float scale = a.sm_scale * kLog2e;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2c, 2c + 1
  float acc[C::MT][4];
#pragma unroll
  for (int i = 0; i < C::MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  for (int p = begin; p < end; p += kTile) {
    const int valid = min(kTile, end - p);
    cp_async_wait<1>();
    __syncwarp();
    float s[4][4];
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j][0] = s[j][1] = s[j][2] = s[j][3] = -INFINITY;
      if (16 * j < valid) {
        float t[4];
        k_job_scores<FMT, D>(kt, kt + O::kCodes, 16 * j + r, qf, ql, corr, lut, c, t);
        if (16 * j + r < valid) {
          s[j][0] = t[0] * scale;
          s[j][1] = t[1] * scale;
        }
        if (16 * j + r + 8 < valid) {
          s[j][2] = t[2] * scale;
          s[j][3] = t[3] * scale;
        }
        x0 = fmaxf(x0, fmaxf(s[j][0], s[j][2]));
        x1 = fmaxf(x1, fmaxf(s[j][1], s[j][3]));
      }
    }
    __syncwarp();  // the K block has been read
    const bool more = p + kTile < end;
    int next = more ? row_of(p + kTile) : 0;
    if (next < 0) next = 0;
    if (more) own_stage<FMT, D>(kt, kc, ks, next, lane);
    cp_async_commit();
#pragma unroll
    for (int o2 = 4; o2 < 32; o2 <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o2));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o2));
    }
    x0 = fmaxf(x0, m0);
    x1 = fmaxf(x1, m1);
    const float f0 = x0 == -INFINITY ? 1.f : ex2(m0 - x0), f1 = x1 == -INFINITY ? 1.f : ex2(m1 - x1);
    m0 = x0;
    m1 = x1;
    l0 *= f0;
    l1 *= f1;
#pragma unroll
    for (int i = 0; i < C::MT; ++i) {
      acc[i][0] *= f0;
      acc[i][1] *= f1;
      acc[i][2] *= f0;
      acc[i][3] *= f1;
    }
    const float b0 = m0 == -INFINITY ? 0.f : kOwnWeightBits - m0, b1 = m1 == -INFINITY ? 0.f : kOwnWeightBits - m1;
    uint32_t p01[4], p89[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float e0 = ex2(s[j][0] + b0), e1 = ex2(s[j][1] + b1), e2 = ex2(s[j][2] + b0), e3 = ex2(s[j][3] + b1);
      l0 += e0 + e2;
      l1 += e1 + e3;
      p01[j] = movmatrix_trans(pack_h2(e0, e1));
      p89[j] = movmatrix_trans(pack_h2(e2, e3));
    }
    cp_async_wait<1>();
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (16 * j < valid) own_v<FMT, D>(vt, vt + O::kCodes, 16 * j, valid, p01[j], p89[j], lane, lut, acc);
    __syncwarp();  // the V block has been read
    if (more) own_stage<FMT, D>(vt, vc, vs, next, lane);
    cp_async_commit();
  }
  cp_async_wait<0>();
#pragma unroll
  for (int o2 = 4; o2 < 32; o2 <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, o2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, o2);
  }
  // heads 2c and 2c + 1 of this lane
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int head = 2 * c + h;
    if (head >= G) continue;
    const int64_t part = ((int64_t)b * a.num_q_heads + kvh * G + head) * o.max_splits + split;
    float* dst = o.part_o + part * D;
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) {
      const int d = C::kQ4 ? 32 * (mt >> 1) + 4 * r + 2 * (mt & 1) : C::kQ8 ? 16 * mt + 2 * r : C::E * r + 2 * mt;
      *reinterpret_cast<float2*>(dst + d) = make_float2(acc[mt][h] * O::kUnhalve, acc[mt][2 + h] * O::kUnhalve);
    }
    if (r == 0) {
      o.part_m[part] = (h ? m1 : m0) - kOwnWeightBits;
      o.part_l[part] = h ? l1 : l0;
    }
  }
}

}  // namespace
}  // namespace kvq
