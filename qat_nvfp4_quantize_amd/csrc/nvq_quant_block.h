// Exact NVFP4 encoding of one 16-element block by one thread, shared by the
// quantizer and the KV-cache writer.  Translation units that include it are
// compiled with -ffp-contract=off: the dequantized value and the residual are
// separately rounded by definition.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvq_device.h"

namespace nvq {

// E4M3 code (0..0x7E) -> fp32.
__device__ __forceinline__ float e4m3_value_f32(uint32_t sc) {
  return (sc >= 8u) ? __uint_as_float((sc + 960u) << 20) : (float)sc * 0x1p-9f;
}

template <int kSel>
__device__ __forceinline__ uint32_t cvt_fp4_pair(uint32_t w, float a, float b) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a, b, 1.0f, kSel);
}

template <int kSel>
__device__ __forceinline__ float2 fp4_pair_to_f32(uint32_t w) {
  auto t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, kSel);
  return make_float2(t[0], t[1]);
}

// Block scale for a tensor scale in the fast range: the E4M3 value nearest the
// real quotient am / (6 s_t), ties to even, saturating at 0x7E (448).
// q = fl(am * g), g = fl(1 / (6 s_t)), is within about 1 ulp of the quotient,
// so it decides alone unless it lies within 8 ulp of an E4M3 midpoint (a
// value with one more significant bit than the grid).  There, the sign of
// am - 6 mid s_t decides: 6 mid has at most 7 significant bits, so
// fma(-(6 mid), s_t, am) rounds the exact difference once and keeps its sign,
// and it is zero exactly on a tie, which goes to the even code.
__device__ __forceinline__ uint32_t e4m3_code_fast(float am, float g, float s_t) {
  const float q = am * g;
  if (!(q < 448.0f)) return 0x7E;
  const uint32_t qb = __float_as_uint(q);
  uint32_t c_lo;
  float mid;
  if (q >= 0.015625f) {
    // normal E4M3: grid = 3 mantissa bits; midpoints have bit 19 set and the
    // low 19 bits clear
    if ((qb & 0xFFFFFu) - 0x80000u + 8u >= 16u)
      return (qb - (120u << 23) + 0x7FFFFu + ((qb >> 20) & 1u)) >> 20;
    mid = __uint_as_float((qb & 0xFFF00000u) | 0x80000u);
    c_lo = ((qb & 0xFFF00000u) - (120u << 23)) >> 20;
  } else {
    // subnormal E4M3: grid 2^-9, midpoints at odd multiples of 2^-10
    const float t = q * 512.0f;
    const float fl = __builtin_floorf(t);
    if (!(fabsf((t - fl) - 0.5f) < 0x1p-16f)) return (uint32_t)__builtin_rintf(t);
    mid = (fl + 0.5f) * 0x1p-9f;
    c_lo = (uint32_t)fl;
  }
  const float d = __builtin_fmaf(-(6.0f * mid), s_t, am);
  return c_lo + ((d > 0.0f || (d == 0.0f && (c_lo & 1u))) ? 1u : 0u);
}

template <bool kBF16>
struct RowBlock {
  uint4 q[kBF16 ? 2 : 4];
  // block blk of row `row` of a tensor whose rows are ld elements apart
  __device__ __forceinline__ void load(const void* xv, int64_t row, int64_t ld, int64_t blk) {
    load_at(static_cast<const char*>(xv) + (row * ld + blk * 16) * (kBF16 ? 2 : 4));
  }
  __device__ __forceinline__ void load_at(const char* at) {
    const uint4* p = reinterpret_cast<const uint4*>(at);
#pragma unroll
    for (int i = 0; i < (kBF16 ? 2 : 4); ++i) q[i] = p[i];
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4& v = q[i >> 2];
    return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
  }
  __device__ __forceinline__ void unpack(float (&xf)[16]) const {
    if (kBF16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xf[2 * j] = bf16_lo(word(j));
        xf[2 * j + 1] = bf16_hi(word(j));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) xf[j] = __uint_as_float(word(j));
    }
  }
  // Stores the raw words into this lane's LDS slot (element j readable by slot_elem).
  __device__ __forceinline__ void to_slot(uint32_t* slot) const {
    uint4* s4 = reinterpret_cast<uint4*>(slot);
#pragma unroll
    for (int i = 0; i < (kBF16 ? 2 : 4); ++i) s4[i] = q[i];
  }
  __device__ static __forceinline__ float slot_elem(const uint32_t* slot, int j) {
    if (kBF16) {
      const uint32_t w = slot[j >> 1];
      return __uint_as_float((j & 1) ? (w & 0xFFFF0000u) : (w << 16));
    }
    return __uint_as_float(slot[j]);
  }
};

// v = fl32(fl32(|G| s_b) s_t) for the 16 codes of a block; acc[j] += |r_j| with
// r_j = fl32(x_j - v_j) (|r| = | |x| - v | since v carries the sign of x).
__device__ __forceinline__ void add_residual(const float (&xf)[16], uint2 cw, float s_b, float s_t,
                                             float (&acc)[16]) {
  float2 g2[8];
  g2[0] = fp4_pair_to_f32<0>(cw.x);
  g2[1] = fp4_pair_to_f32<1>(cw.x);
  g2[2] = fp4_pair_to_f32<2>(cw.x);
  g2[3] = fp4_pair_to_f32<3>(cw.x);
  g2[4] = fp4_pair_to_f32<0>(cw.y);
  g2[5] = fp4_pair_to_f32<1>(cw.y);
  g2[6] = fp4_pair_to_f32<2>(cw.y);
  g2[7] = fp4_pair_to_f32<3>(cw.y);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v0 = (fabsf(g2[j].x) * s_b) * s_t;
    const float v1 = (fabsf(g2[j].y) * s_b) * s_t;
    acc[2 * j] += fabsf(fabsf(xf[2 * j]) - v0);
    acc[2 * j + 1] += fabsf(fabsf(xf[2 * j + 1]) - v1);
  }
}

// One block, tensor scale in the fast range.  Element codes: the hardware FP4
// conversion rounds y = x h with h bracketed at (1 -+ 2^-20) / (s_b s_t); y is
// within 2^-21.5 of the real quotient, so both brackets agree unless the
// quotient is within 2^-19 of an E2M1 midpoint.  Where they disagree the
// upper index is the lower plus one and the sign of |x| - m s_b s_t (m the
// midpoint between them; m s_b has at most 7 significant bits, so one fma
// rounds the exact difference once) decides; zero is a tie, which goes to the
// even index.  slot: this lane's LDS words for the rare fix-up.
template <bool kBF16, bool kScore>
__device__ __forceinline__ void encode_block_fast(const RowBlock<kBF16>& rb, float s_t, float g,
                                                  float inv_st, uint32_t& sc_out, uint2& cw_out,
                                                  float (&acc)[16], uint32_t& bad, uint32_t* slot) {
  float xf[16];
  rb.unpack(xf);
  float am = __builtin_fmaxf(__builtin_fmaxf(fabsf(xf[0]), fabsf(xf[1])), fabsf(xf[2]));
#pragma unroll
  for (int j = 3; j < 15; j += 2) am = __builtin_fmaxf(__builtin_fmaxf(am, fabsf(xf[j])), fabsf(xf[j + 1]));
  am = __builtin_fmaxf(am, fabsf(xf[15]));
  if (!(am <= 3.40282347e38f)) bad = 1;
  const uint32_t sc = e4m3_code_fast(am, g, s_t);
  sc_out = sc;
  const float s_b = e4m3_value_f32(sc);
  const float h = sc == 0 ? 0.0f : __builtin_amdgcn_rcpf(s_b) * inv_st;
  const float h_lo = h * 0.99999904632568359375f;  // 1 - 2^-20
  const float h_hi = h * 1.00000095367431640625f;  // 1 + 2^-20
  uint32_t lo0 = 0, lo1 = 0, hi0 = 0, hi1 = 0;
  lo0 = cvt_fp4_pair<0>(lo0, xf[0] * h_lo, xf[1] * h_lo);
  lo0 = cvt_fp4_pair<1>(lo0, xf[2] * h_lo, xf[3] * h_lo);
  lo0 = cvt_fp4_pair<2>(lo0, xf[4] * h_lo, xf[5] * h_lo);
  lo0 = cvt_fp4_pair<3>(lo0, xf[6] * h_lo, xf[7] * h_lo);
  lo1 = cvt_fp4_pair<0>(lo1, xf[8] * h_lo, xf[9] * h_lo);
  lo1 = cvt_fp4_pair<1>(lo1, xf[10] * h_lo, xf[11] * h_lo);
  lo1 = cvt_fp4_pair<2>(lo1, xf[12] * h_lo, xf[13] * h_lo);
  lo1 = cvt_fp4_pair<3>(lo1, xf[14] * h_lo, xf[15] * h_lo);
  hi0 = cvt_fp4_pair<0>(hi0, xf[0] * h_hi, xf[1] * h_hi);
  hi0 = cvt_fp4_pair<1>(hi0, xf[2] * h_hi, xf[3] * h_hi);
  hi0 = cvt_fp4_pair<2>(hi0, xf[4] * h_hi, xf[5] * h_hi);
  hi0 = cvt_fp4_pair<3>(hi0, xf[6] * h_hi, xf[7] * h_hi);
  hi1 = cvt_fp4_pair<0>(hi1, xf[8] * h_hi, xf[9] * h_hi);
  hi1 = cvt_fp4_pair<1>(hi1, xf[10] * h_hi, xf[11] * h_hi);
  hi1 = cvt_fp4_pair<2>(hi1, xf[12] * h_hi, xf[13] * h_hi);
  hi1 = cvt_fp4_pair<3>(hi1, xf[14] * h_hi, xf[15] * h_hi);
  uint32_t d0 = lo0 ^ hi0, d1 = lo1 ^ hi1;
  if (d0 | d1) {
    rb.to_slot(slot);
    const float half_sb = 0.5f * s_b;
#pragma unroll 1
    while (d0 | d1) {
      const bool first = d0 != 0;
      const uint32_t sh = __builtin_ctz(first ? d0 : d1) & ~3u;
      const int j = (first ? 0 : 8) + (int)(sh >> 2);
      const uint32_t wl = first ? lo0 : lo1;
      const uint32_t il = (wl >> sh) & 7u, ih = ((first ? hi0 : hi1) >> sh) & 7u;
      // |G_lo| and |G_hi| from one conversion of the byte (il, ih)
      const float2 gg = fp4_pair_to_f32<0>(il | (ih << 4));
      const float d = __builtin_fmaf(-((gg.x + gg.y) * half_sb), s_t,
                                     fabsf(RowBlock<kBF16>::slot_elem(slot, j)));
      const uint32_t pick = (d > 0.0f || (d == 0.0f && !(ih & 1u))) ? ih : il;
      const uint32_t nw = (wl & ~(7u << sh)) | (pick << sh);
      if (first) {
        lo0 = nw;
        d0 &= ~(15u << sh);
      } else {
        lo1 = nw;
        d1 &= ~(15u << sh);
      }
    }
  }
  cw_out = make_uint2(lo0, lo1);
  if (kScore) add_residual(xf, cw_out, s_b, s_t, acc);
}

// One block decided entirely in fp64 (tensor scale outside [2^-100, 2^100],
// where the fp32 reciprocals would overflow).  Off the hot path.
template <bool kBF16, bool kScore>
__device__ __forceinline__ void encode_block_exact(const RowBlock<kBF16>& rb, float s_t,
                                                   double six_st, uint32_t& sc_out,
                                                   uint2& cw_out, float (&acc)[16],
                                                   uint32_t& bad, uint32_t* slot) {
  float xf[16];
  rb.unpack(xf);
  float am = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) am = __builtin_fmaxf(am, fabsf(xf[j]));
  if (!(am <= 3.40282347e38f)) bad = 1;
  const uint32_t sc = s_t > 0.0f ? e4m3_code_exact(am, six_st) : 0u;
  sc_out = sc;
  const float s_b = e4m3_value_f32(sc);
  rb.to_slot(slot);
  const double S = (double)s_b * (double)s_t;
  uint32_t c0 = 0u, c1 = 0u;
#pragma unroll 1
  for (int j = 0; j < 16; ++j) {
    const float v = RowBlock<kBF16>::slot_elem(slot, j);
    const uint32_t idx = (sc == 0) ? 0u : e2m1_index_exact(fabsf(v), S);
    const uint32_t nib = (idx | ((__float_as_uint(v) >> 28) & 8u)) << (4 * (j & 7));
    c0 |= (j < 8) ? nib : 0u;
    c1 |= (j < 8) ? 0u : nib;
  }
  cw_out = make_uint2(c0, c1);
  if (kScore) add_residual(xf, cw_out, s_b, s_t, acc);
}

// v_j = sign * fl32(fl32(G s_b) s_t) of the 16 codes of a block.
__device__ __forceinline__ void block_values(uint2 cw, float s_b, float s_t, float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w = h ? cw.y : cw.x;
    float2 g[4];
    g[0] = fp4_pair_to_f32<0>(w);
    g[1] = fp4_pair_to_f32<1>(w);
    g[2] = fp4_pair_to_f32<2>(w);
    g[3] = fp4_pair_to_f32<3>(w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * h + 2 * j] = (g[j].x * s_b) * s_t;
      v[8 * h + 2 * j + 1] = (g[j].y * s_b) * s_t;
    }
  }
}

// Stores 16 values as bf16 (32 bytes) or fp32 (64 bytes).
template <bool kBF16>
__device__ __forceinline__ void store_block(const float (&v)[16], void* at) {
  if (kBF16) {
    uint4* o = static_cast<uint4*>(at);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float* u = v + 8 * q;
      o[q] = make_uint4(f32_to_bf16_rne(u[0]) | (f32_to_bf16_rne(u[1]) << 16),
                        f32_to_bf16_rne(u[2]) | (f32_to_bf16_rne(u[3]) << 16),
                        f32_to_bf16_rne(u[4]) | (f32_to_bf16_rne(u[5]) << 16),
                        f32_to_bf16_rne(u[6]) | (f32_to_bf16_rne(u[7]) << 16));
    }
  } else {
    float4* o = static_cast<float4*>(at);
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  }
}

}  // namespace nvq
