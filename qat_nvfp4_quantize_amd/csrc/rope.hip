// Rotary positions of projected heads, both pair layouts, forward and
// gradient, and the host-side frequency tables.
//
// Mathematics: pair (u, w) of token t turns by the angle positions[t] f_j.
// The angle is taken as turns, positions[t] * (f_j / 2 pi) in fp64, reduced
// to [-1/2, 1/2] there and only then rounded to fp32, so far positions lose
// nothing (an fp32 product is off by 2^-24 of the angle, 0.008 radians at
// position 131072).  Sine and cosine depend on (token, pair) only: a
// workgroup computes them once into LDS for all its heads.  From the rounded
// half turns on everything is fp32 (sine and cosine within 2 steps): an fp32
// result's relative rms error is 6.2e-8 against 4.6e-8 from 64-bit sines, at
// half a step of 6.0e-8; a bf16 result's is the same.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "nvq.h"
#include "nvq_device.h"
#include "nvq_internal.h"

namespace nvq {
namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
  const char* x;
  char* y;
  int64_t x_ld_t, x_ld_h, y_ld_t, y_ld_h;  // elements
  const int32_t* positions;
  const double* inv_freq;
  int64_t T;
  int H, D, rot;
  int copy_rest;  // elements past rot are copied (y != x)
  int tt, hc;     // tokens and heads of a workgroup
  float mag, sign;
};

// One 16-byte vector of elements as fp32.
template <bool kBF16>
struct RopeVec {
  static constexpr int kN = kBF16 ? 8 : 4;
  float v[kN];
  __device__ __forceinline__ void unpack(uint4 q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kBF16) {
        v[2 * i] = bf16_lo(w[i]);
        v[(2 * i + 1) % kN] = bf16_hi(w[i]);
      } else {
        v[i] = __uint_as_float(w[i]);
      }
    }
  }
  __device__ __forceinline__ void store(char* at) const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = kBF16 ? f32_to_bf16_any(v[(2 * i) % kN]) | (f32_to_bf16_any(v[(2 * i + 1) % kN]) << 16)
                   : __float_as_uint(v[i]);
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// kVec: 16-byte vectors of a row's elements (half layout: a vector of each
// half; interleaved: a vector of whole pairs; then the copied rest), else
// single pairs (any size, stride and element alignment).  HBM-bound: every
// element is read and written once.
template <bool kBF16, bool kInter, bool kVec>
__global__ __launch_bounds__(kRopeThreads) void k_rope(RopeParams p) {
  extern __shared__ float2 s_cs[];  // [tt][rot / 2] (m cos, +-m sin)
  constexpr int kSize = kBF16 ? 2 : 4;
  constexpr int kN = kVec ? RopeVec<kBF16>::kN : 1;
  const int half = p.rot >> 1;
  const int64_t t0 = (int64_t)blockIdx.x * p.tt;
  const int tn = (int)min<int64_t>(p.tt, p.T - t0);
  for (int i = threadIdx.x; i < tn * half; i += kRopeThreads) {
    const int tok = i / half, j = i - tok * half;
    const double turns = (double)p.positions[t0 + tok] * (p.inv_freq[j] * 0.15915494309189533577);
    const float r = (float)(2.0 * (turns - rint(turns)));
    float sn, cs;
    sincospif(r, &sn, &cs);
    s_cs[i] = make_float2(cs * p.mag, sn * p.mag * p.sign);
  }
  __syncthreads();
  const int h0 = blockIdx.y * p.hc, hn = min(p.hc, p.H - h0);
  if constexpr (!kVec) {
    const int per_row = half + (p.copy_rest ? p.D - p.rot : 0);
    for (int it = threadIdx.x; it < tn * hn * per_row; it += kRopeThreads) {
      const int row = it / per_row, c = it - row * per_row, tok = row / hn;
      const int64_t t = t0 + tok, h = h0 + (row - tok * hn);
      using Elem = std::conditional_t<kBF16, uint16_t, float>;
      const Elem* xr = reinterpret_cast<const Elem*>(p.x) + t * p.x_ld_t + h * p.x_ld_h;
      Elem* yr = reinterpret_cast<Elem*>(p.y) + t * p.y_ld_t + h * p.y_ld_h;
      if (c >= half) {
        yr[p.rot + c - half] = xr[p.rot + c - half];
        continue;
      }
      const int u = kInter ? 2 * c : c, w = kInter ? 2 * c + 1 : c + half;
      const float2 q = s_cs[tok * half + c];
      if constexpr (kBF16) {
        const float a = bf16_to_f32(xr[u]), b = bf16_to_f32(xr[w]);
        yr[u] = (uint16_t)f32_to_bf16_any(a * q.x - b * q.y);
        yr[w] = (uint16_t)f32_to_bf16_any(a * q.y + b * q.x);
      } else {
        const float a = xr[u], b = xr[w];
        yr[u] = a * q.x - b * q.y;
        yr[w] = a * q.y + b * q.x;
      }
    }
  } else {
    // A thread keeps its vector c of the row (two of them in the half layout)
    // and walks the rows, kAtOnce of them loaded before the first is stored.
    constexpr int kAtOnce = kInter ? 4 : 2;
    const int n_rot = (kInter ? p.rot : half) / kN, per_row = n_rot + (p.copy_rest ? (p.D - p.rot) / kN : 0);
    const int lanes = min(per_row, kRopeThreads), step = kRopeThreads / lanes;
    const int first = threadIdx.x / lanes;
    if (first >= step) return;  // threads past the last whole row
    for (int c = threadIdx.x - first * lanes; c < per_row; c += lanes) {
      const bool turn = c < n_rot;
      const int64_t at = turn ? (int64_t)c * 16 : (int64_t)p.rot * kSize + (int64_t)(c - n_rot) * 16;
      const int64_t second = (int64_t)half * kSize;
      int tok = first / hn, h = first - tok * hn;
      while (tok < tn) {
        uint4 a[kAtOnce], b[kAtOnce];
        int rt[kAtOnce], rh[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          rt[i] = tok, rh[i] = h0 + h;
          if (tok < tn) {
            const char* xr = p.x + ((t0 + tok) * p.x_ld_t + rh[i] * p.x_ld_h) * kSize + at;
            a[i] = *reinterpret_cast<const uint4*>(xr);
            if (!kInter && turn) b[i] = *reinterpret_cast<const uint4*>(xr + second);
          }
          h += step;
          while (h >= hn) h -= hn, ++tok;
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          if (rt[i] >= tn) break;
          char* yr = p.y + ((t0 + rt[i]) * p.y_ld_t + rh[i] * p.y_ld_h) * kSize + at;
          if (!turn) {
            *reinterpret_cast<uint4*>(yr) = a[i];
            continue;
          }
          const float2* cs = s_cs + rt[i] * half + (kInter ? c * (kN / 2) : c * kN);
          RopeVec<kBF16> u;
          u.unpack(a[i]);
          if constexpr (kInter) {
#pragma unroll
            for (int j = 0; j < kN; j += 2) {
              const float2 q = cs[j / 2];
              const float m = u.v[j], n = u.v[j + 1];
              u.v[j] = m * q.x - n * q.y;
              u.v[j + 1] = m * q.y + n * q.x;
            }
          } else {
            RopeVec<kBF16> w;
            w.unpack(b[i]);
#pragma unroll
            for (int j = 0; j < kN; ++j) {
              const float2 q = cs[j];
              const float m = u.v[j], n = w.v[j];
              u.v[j] = m * q.x - n * q.y;
              w.v[j] = m * q.y + n * q.x;
            }
            w.store(yr + second);
          }
          u.store(yr);
        }
      }
    }
  }
}

template <bool kBF16, bool kInter>
void launch_rope(const RopeParams& p, bool vec, dim3 grid, size_t lds, hipStream_t s) {
  if (vec)
    hipLaunchKernelGGL((k_rope<kBF16, kInter, true>), grid, dim3(kRopeThreads), lds, s, p);
  else
    hipLaunchKernelGGL((k_rope<kBF16, kInter, false>), grid, dim3(kRopeThreads), lds, s, p);
}

}  // namespace
}  // namespace nvq

using namespace nvq;

extern "C" int nvq_rope(const void* x, int dtype, int64_t T, int64_t H, int64_t D, int64_t x_ld_t,
                        int64_t x_ld_h, const int32_t* positions, const double* inv_freq,
                        int64_t rot_dim, int layout, float magnitude, int inverse, void* y,
                        int64_t y_ld_t, int64_t y_ld_h, void* stream) {
  if (dtype != NVQ_F32 && dtype != NVQ_BF16) return NVQ_EINVAL;
  if (layout != NVQ_ROPE_HALF && layout != NVQ_ROPE_INTERLEAVED) return NVQ_EINVAL;
  if (T < 0 || T > kMaxTokens || H < 0 || H > 65535 || D < 2 || D > 4096 || rot_dim < 2 || rot_dim > D ||
      (rot_dim & 1))
    return NVQ_ESHAPE;
  if (x_ld_t == 0) x_ld_t = H * D;
  if (x_ld_h == 0) x_ld_h = D;
  if (y_ld_t == 0) y_ld_t = H * D;
  if (y_ld_h == 0) y_ld_h = D;
  if (x_ld_t < 0 || x_ld_h < 0 || y_ld_t < 0 || y_ld_h < 0) return NVQ_ESHAPE;
  if (T == 0 || H == 0) return NVQ_OK;
  // rows of y must not overlap
  if ((H > 1 && y_ld_h < D) || (T > 1 && y_ld_t < D)) return NVQ_ESHAPE;
  if (H > 1 && T > 1 && y_ld_t < (H - 1) * y_ld_h + D && y_ld_h < (T - 1) * y_ld_t + D) return NVQ_ESHAPE;
  if (!x || !y || !positions || !inv_freq) return NVQ_EINVAL;
  if (x == y && (x_ld_t != y_ld_t || x_ld_h != y_ld_h)) return NVQ_EINVAL;
  const int size = dtype == NVQ_BF16 ? 2 : 4, n = 16 / size;
  if (((uintptr_t)x | (uintptr_t)y) % size || ((uintptr_t)positions & 3u) || ((uintptr_t)inv_freq & 7u))
    return NVQ_EALIGN;
  RopeParams p{};
  p.x = static_cast<const char*>(x);
  p.y = static_cast<char*>(y);
  p.x_ld_t = x_ld_t, p.x_ld_h = x_ld_h, p.y_ld_t = y_ld_t, p.y_ld_h = y_ld_h;
  p.positions = positions, p.inv_freq = inv_freq;
  p.T = T, p.H = (int)H, p.D = (int)D, p.rot = (int)rot_dim;
  p.copy_rest = x != y;
  p.mag = magnitude;
  p.sign = inverse ? -1.0f : 1.0f;
  const bool vec = aligned16(x) && aligned16(y) && rot_dim % (2 * n) == 0 && D % n == 0 && x_ld_t % n == 0 &&
                   x_ld_h % n == 0 && y_ld_t % n == 0 && y_ld_h % n == 0;
  const bool inter = layout == NVQ_ROPE_INTERLEAVED;
  const int half = p.rot / 2, step = vec ? n : 1;
  const int64_t per_row = (inter && vec ? p.rot : half) / step + (p.copy_rest ? (p.D - p.rot) / step : 0);
  // Up to 16 vectors a thread, fewer where that leaves CUs without a
  // workgroup: a workgroup takes the sines of its tokens anew, which at 4
  // vectors cost as much as the rotation (8192 x 40 x 128 bf16, 64 elements
  // turned: 44 us against 38; a copy of the tensor 33).
  const int64_t per_wg =
      std::clamp<int64_t>(T * H * per_row / (4 * (int64_t)device_cu_count()), kRopeThreads, 16 * kRopeThreads);
  p.tt = (int)std::clamp<int64_t>(kRopeThreads / half, 1, std::min<int64_t>(16, T));
  p.hc = (int)std::clamp<int64_t>(per_wg / (p.tt * per_row), 1, H);
  const int64_t gx = (T + p.tt - 1) / p.tt, gy = (H + p.hc - 1) / p.hc;
  const dim3 grid((unsigned)gx, (unsigned)gy);
  const size_t lds = (size_t)p.tt * half * sizeof(float2);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == NVQ_BF16) {
    if (inter) launch_rope<true, true>(p, vec, grid, lds, s);
    else launch_rope<true, false>(p, vec, grid, lds, s);
  } else {
    if (inter) launch_rope<false, true>(p, vec, grid, lds, s);
    else launch_rope<false, false>(p, vec, grid, lds, s);
  }
  return last_launch();
}

extern "C" int nvq_rope_frequencies(int kind, int64_t rot_dim, double base, double factor, double orig_len,
                                    double slow, double fast, double* inv_freq, float* magnitude) {
  if (!inv_freq || kind < NVQ_ROPE_PLAIN || kind > NVQ_ROPE_RAMP) return NVQ_EINVAL;
  if (rot_dim < 2 || (rot_dim & 1) || rot_dim > 4096) return NVQ_ESHAPE;
  if (!(base > 0.0) || !std::isfinite(base)) return NVQ_EINVAL;
  if (kind != NVQ_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return NVQ_EINVAL;
  if (kind == NVQ_ROPE_BASE) {
    if (!(base > 1.0)) return NVQ_EINVAL;
    if (rot_dim < 4) return NVQ_ESHAPE;
    base *= std::pow(factor, (double)rot_dim / (double)(rot_dim - 2));
  }
  if (kind == NVQ_ROPE_RAMP &&
      (!(orig_len > 0.0) || !std::isfinite(orig_len) || !(slow > 0.0) || !(fast > slow) || !std::isfinite(fast)))
    return NVQ_EINVAL;
  for (int64_t j = 0; j < rot_dim / 2; ++j) {
    double f = std::pow(base, -2.0 * (double)j / (double)rot_dim);
    if (kind == NVQ_ROPE_LINEAR) f /= factor;
    if (kind == NVQ_ROPE_RAMP) {
      const double turns = orig_len * f / 6.28318530717958647693;
      const double r = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
      f = f * r + f / factor * (1.0 - r);
    }
    inv_freq[j] = f;
  }
  if (magnitude) *magnitude = kind == NVQ_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return NVQ_OK;
}
