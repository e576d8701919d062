// Root-mean-square norm with the residual's addition, forward (bf16 / fp32 or
// 8-bit output) and gradient.
//
//   h = round(x + residual),  r = (mean h^2 + eps)^(-1/2),  y = h r weight
//   E4M3: s_g = max(max|y| / 448, 2^-126) per group, code = e4m3(y / s_g)
//   dx = r (g - u mean(g u)) + dh with g = dy weight, u = h r
//   dweight = sum over rows of dy u
//
// Bound by HBM: a row stays in registers between its two passes, so each
// tensor moves once (16384 rows of 4096 bf16 with a residual 88 to 91 us, 6 TB/s;
// the gradient with dh 104 to 114 us, 5 TB/s, and 5 to join dweight; 32768 rows
// into E4M3 180 us, 5.2 TB/s, in groups of 32, 64 or 128 alike, with one scale a
// row 199).  The sum of squares is fp64 (a conversion and an fma per element, far
// below what the loads leave room for), so no row of finite values overflows or
// vanishes in it.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "nvq.h"
#include "nvq_device.h"
#include "nvq_internal.h"

namespace nvq {
namespace {

constexpr int kMaxD = 32768;

// Values of the lane that a DPP step pairs this one with, inside rows of 16:
// 0xB1 quad_perm [1,0,3,2], 0x4E quad_perm [2,3,0,1], 0x141 row_half_mirror,
// 0x140 row_mirror.  One after the other they join 2, 4, 8 and 16 lanes.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, kCtrl, 0xF, 0xF, false);
}
template <int kCtrl>
__device__ __forceinline__ uint64_t dpp(uint64_t v) {
  return ((uint64_t)dpp<kCtrl>((uint32_t)(v >> 32)) << 32) | dpp<kCtrl>((uint32_t)v);
}
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<kCtrl>(__float_as_uint(v)));
}
template <int kCtrl>
__device__ __forceinline__ double dpp(double v) {
  return __longlong_as_double((long long)dpp<kCtrl>((uint64_t)__double_as_longlong(v)));
}

// A row belongs to kL lanes (of one wave, or whole waves of a workgroup), which
// hold kN vectors of 8 elements each.
template <int kL>
struct Group {
  static constexpr int kThreads = kL <= 64 ? 256 : kL;
  static constexpr int kLanes = kL, kRows = kThreads / kL, kWaves = kL <= 64 ? 1 : kL / 64;
  __device__ static __forceinline__ int lane() { return threadIdx.x & (kL - 1); }
  __device__ static __forceinline__ int row() { return kRows > 1 ? (int)threadIdx.x / kL : 0; }
  template <class T, class F>
  __device__ static __forceinline__ T join(T v, F&& f) {
    v = f(v, dpp<0xB1>(v));
    v = f(v, dpp<0x4E>(v));
    if (kL >= 8) v = f(v, dpp<0x141>(v));
    if (kL >= 16) v = f(v, dpp<0x140>(v));
    if (kL >= 32) v = f(v, (T)__shfl_xor(v, 16, 64));
    if (kL >= 64) v = f(v, (T)__shfl_xor(v, 32, 64));
    return v;
  }
  // s: one slot a wave, not in use by an earlier reduction
  template <class T>
  __device__ static __forceinline__ T sum(T v, T* s) {
    v = join(v, [](T a, T b) { return a + b; });
    if (kWaves == 1) return v;
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0] + s[1];
#pragma unroll
    for (int i = 2; i < kWaves; i += 2) v += s[i] + s[i + 1];
    return v;
  }
  // Maximum of non-negative values as bit patterns, where a NaN is the largest.
  template <class T>
  __device__ static __forceinline__ T top(T v, T* s) {
    v = join(v, [](T a, T b) { return max(a, b); });
    if (kWaves == 1) return v;
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v = max(v, s[i]);
    return v;
  }
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Eight consecutive elements of a bf16 or fp32 row.
template <bool kBF16>
struct Vec;
template <>
struct Vec<true> {
  u32x4 q;
  __device__ __forceinline__ void clear() { q = 0u; }
  // the same bits as a value that nothing earlier is known of
  __device__ __forceinline__ Vec anew() const {
    Vec v = *this;
    asm volatile("" : "+v"(v.q));
    return v;
  }
  __device__ __forceinline__ void load(const void* row, int v) { q = static_cast<const u32x4*>(row)[v]; }
  __device__ __forceinline__ void store(void* row, int v) const { static_cast<u32x4*>(row)[v] = q; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (j & 1) ? bf16_hi(q[j >> 1]) : bf16_lo(q[j >> 1]);
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = pack_bf16(f[2 * j], f[2 * j + 1]);
  }
};
template <>
struct Vec<false> {
  u32x4 a, b;
  __device__ __forceinline__ void clear() { a = b = 0u; }
  __device__ __forceinline__ Vec anew() const {
    Vec v = *this;
    asm volatile("" : "+v"(v.a), "+v"(v.b));
    return v;
  }
  __device__ __forceinline__ void load(const void* row, int v) {
    a = static_cast<const u32x4*>(row)[2 * v];
    b = static_cast<const u32x4*>(row)[2 * v + 1];
  }
  __device__ __forceinline__ void store(void* row, int v) const {
    static_cast<u32x4*>(row)[2 * v] = a;
    static_cast<u32x4*>(row)[2 * v + 1] = b;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = __uint_as_float(a[j]);
      f[4 + j] = __uint_as_float(b[j]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = __float_as_uint(f[j]);
      b[j] = __float_as_uint(f[4 + j]);
    }
  }
};

struct NormParams {
  int64_t T, D, x_ld, res_ld, h_ld, y_ld;
  const void* x;
  const void* res;
  const void* weight;
  double eps;
  void* h;
  void* y;
  uint8_t* y8;
  float* scales;
  int group;
  float* rstd;
  uint32_t* amax;
};

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// The E4M3 output is decided as the real quotients 448 y / max|y| are.  An fp32
// quotient is off by at most 8 roundings (3 of y, 4 of the scale's inverse, its
// own), so it decides alone unless it lies within 10 ulp of a midpoint of the
// format; those are decided again in fp64 from 448 h w / max|h w|, the same
// number with exact products, so that a tie is a tie (with bf16 rows and weights
// about one element in 3000 is one).  32768 rows of 4096 took 181 us when this
// was built, without the second decision 161, with every one in fp64 208.

// The scale of a group whose largest |y| has these bits, and 1 / it.  A NaN
// stays one (a maximum alone would drop it).
struct Scale {
  float stored, inverse;
};
constexpr float kLeastScale = 0x1p-126f;
__device__ __forceinline__ Scale scale_of(uint32_t bits) {
  const float top = __uint_as_float(bits);
  if (!(top == top)) return {top, top};
  if (top < 448.0f * kLeastScale) return {kLeastScale, 0x1p126f};
  return {top / 448.0f, 448.0f / top};
}

// Whether q is so near a midpoint that its last bits matter.  Midpoints of the
// normal numbers have the 20 low bits 0x80000; below 2^-6 the format's step is
// that of the binade above, which adding 2^-6 moves q into.
__device__ __forceinline__ bool near_midpoint(float q) {
  const float a = fabsf(q), w = a < 0x1p-6f ? a + 0x1p-6f : a;
  return (__float_as_uint(w) & 0xFFFFFu) - (0x80000u - 10u) <= 20u;
}

// q cut to fp32 with its lowest bit set where anything was cut off: it rounds to
// E4M3 as q itself does.  Below 2^-20 it is zero, as it rounds to.
__device__ __forceinline__ float cut(double q) {
  const uint64_t b = (uint64_t)__double_as_longlong(q);
  const uint32_t sign = (uint32_t)(b >> 32) & 0x80000000u;
  const uint64_t mag = b & 0x7FFFFFFFFFFFFFFFull;
  if (mag < 0x3EB0000000000000ull) return __uint_as_float(sign);
  const uint32_t m = (uint32_t)((mag - 0x3800000000000000ull) >> 29);
  return __uint_as_float(sign | m | (((uint32_t)b & 0x1FFFFFFFu) != 0u ? 1u : 0u));
}

__device__ __forceinline__ void store_e4m3(uint8_t* at, const float (&q)[8]) {
  uint32_t lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  *reinterpret_cast<uint2*>(at) = make_uint2(lo, hi);
}

// Magnitudes of fp64 values are compared as bit patterns, where a NaN is the largest.
__device__ __forceinline__ uint64_t magnitude(double f) { return (uint64_t)__double_as_longlong(f) & 0x7FFFFFFFFFFFFFFFull; }

// Maximum over the 4, 8 or 16 neighbouring lanes of a group.
template <class T>
__device__ __forceinline__ T group_top(T m, int lanes) {
  m = max(m, dpp<0xB1>(m));
  m = max(m, dpp<0x4E>(m));
  if (lanes > 4) m = max(m, dpp<0x141>(m));
  if (lanes > 8) m = max(m, dpp<0x140>(m));
  return m;
}

// kOut: 0 y alone, 1 also (or only) 8 bits with scales of groups, 2 with one of the row
template <bool kBF16, bool kWBF16, int kOut, int kL, int kN>
__global__ __launch_bounds__(Group<kL>::kThreads) void k_rms_norm(NormParams p) {
  using G = Group<kL>;
  __shared__ double s_sum[G::kWaves];
  __shared__ uint64_t s_product[G::kWaves];
  __shared__ uint32_t s_max[G::kWaves], s_amax[G::kWaves];
  const int size = kBF16 ? 2 : 4;
  const int nvec = (int)(p.D / 8), lane = G::lane();
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * G::kRows + G::row();
  if (t >= p.T) return;  // a whole workgroup, or lanes that share none with other rows, where no barrier follows
  const char* const xr = static_cast<const char*>(p.x) + t * p.x_ld * size;
  Vec<kBF16> x[kN];
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int v = lane + k * G::kLanes;
    x[k].clear();
    if (v < nvec) x[k].load(xr, v);
  }
  if (p.res) {
    const char* const rr = static_cast<const char*>(p.res) + t * p.res_ld * size;
    char* const hr = static_cast<char*>(p.h) + t * p.h_ld * size;
    Vec<kBF16> r[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k)
      if (lane + k * G::kLanes < nvec) r[k].load(rr, lane + k * G::kLanes);
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int v = lane + k * G::kLanes;
      if (v >= nvec) continue;
      float a[8], b[8];
      x[k].get(a);
      r[k].get(b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] += b[j];
      x[k].set(a);
      x[k].store(hr, v);
    }
  }
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    float a[8];
    x[k].get(a);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)a[j], (double)a[j], sum);
  }
  sum = G::sum(sum, s_sum);
  const float r = (float)(1.0 / sqrt(sum / (double)p.D + p.eps));
  if (p.rstd && lane == 0) p.rstd[t] = r;
  // h and weight of this lane's k-th vector, y of it, and the largest |h w|.  Each
  // unpacks the row again: kept unpacked (in fp64, after the sum of squares) it
  // would take twice the registers, and half the waves would be resident.
  auto factors = [&](int k, float (&h)[8], float (&w)[8]) {
    Vec<kWBF16> wv;
    wv.load(p.weight, lane + k * G::kLanes);
    wv.get(w);
    x[k].anew().get(h);
  };
  auto values = [&](int k, float (&f)[8]) {
    float w[8];
    factors(k, f, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * r * w[j];
  };
  auto largest_product = [&](int k) -> uint64_t {
    float h[8], w[8];
    factors(k, h, w);
    uint64_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, magnitude((double)h[j] * (double)w[j]));
    return m;
  };
  // decides the marked codes of a vector again; few lanes have any
  auto decide = [&](int k, uint32_t marked, uint64_t largest) {
    const int v = lane + k * G::kLanes;
    const double d = __longlong_as_double((long long)largest);
    while (marked) {
      const int j = __builtin_ctz(marked);
      marked &= marked - 1;
      float h[8], hj = 0.0f;
      x[k].anew().get(h);
#pragma unroll
      for (int i = 0; i < 8; ++i) hj = i == j ? h[i] : hj;
      const int64_t at = 8 * (int64_t)v + j;
      const float w = kWBF16 ? bf16_to_f32(static_cast<const uint16_t*>(p.weight)[at]) : static_cast<const float*>(p.weight)[at];
      const float q = cut(448.0 * ((double)hj * (double)w) / d);
      p.y8[t * p.D + at] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false);
    }
  };
  uint32_t top = 0, row_top = 0;
  uint64_t row_product = 0;
  constexpr bool k8 = kOut != 0, whole = kOut == 2;
  const int lanes = p.group / 8;  // lanes that share a group: 4, 8 or 16 in a row
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int v = lane + k * G::kLanes;
    float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (v < nvec) values(k, f);
    if (p.y && v < nvec) {
      Vec<kBF16> o;
      o.set(f);
      o.store(static_cast<char*>(p.y) + t * p.y_ld * size, v);
      if (p.amax) {
        float q[8];
        o.get(q);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, abs_bits(q[j]));
      }
    }
    if (!k8) continue;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(f[j]));
    if (whole) {
      row_top = max(row_top, m);
      if (v < nvec) row_product = max(row_product, largest_product(k));
      continue;
    }
    const Scale s = scale_of(group_top(m, lanes));
    uint32_t again = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] *= s.inverse;
      again |= near_midpoint(f[j]) ? 1u << j : 0u;
    }
    if (!(s.stored > kLeastScale)) again = 0;  // nor a NaN's: its low bits mean nothing
    if (v < nvec) {
      if (v % lanes == 0) p.scales[t * (p.D / p.group) + v / lanes] = s.stored;
      store_e4m3(p.y8 + t * p.D + 8 * (int64_t)v, f);
    }
    if (__any(again != 0)) decide(k, again, group_top(v < nvec ? largest_product(k) : (uint64_t)0, lanes));
  }
  if (whole) {
    const Scale s = scale_of(G::top(row_top, s_max));
    row_product = G::top(row_product, s_product);
    if (lane == 0) p.scales[t] = s.stored;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int v = lane + k * G::kLanes;
      if (v >= nvec) continue;
      float f[8];
      values(k, f);
      uint32_t again = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[j] *= s.inverse;
        again |= near_midpoint(f[j]) ? 1u << j : 0u;
      }
      store_e4m3(p.y8 + t * p.D + 8 * (int64_t)v, f);
      if (s.stored > kLeastScale) decide(k, again, row_product);
    }
  }
  if (p.amax) {
    top = G::top(top, s_amax);
    if (lane == 0 && top > __hip_atomic_load(p.amax, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(p.amax, top);
  }
}

__global__ void k_zero_word(uint32_t* w) { *w = 0u; }

struct NormGradParams {
  int64_t T, D, dy_ld, h_ld, dh_ld, dx_ld;
  const void* dy;
  const void* h;
  const void* weight;
  const float* rstd;
  const void* dh;
  void* dx;
  float* part;  // [workgroups, D], NULL: no dweight
};

template <bool kBF16, bool kWBF16, int kL, int kN>
__global__ __launch_bounds__(Group<kL>::kThreads) void k_rms_grad(NormGradParams p) {
  using G = Group<kL>;
  __shared__ float s_sum[2][G::kWaves];
  const int size = kBF16 ? 2 : 4;
  const int nvec = (int)(p.D / 8), lane = G::lane(), unit = blockIdx.x * G::kRows + G::row();
  const float inv_d = 1.0f / (float)p.D;
  float acc[kN][8];
#pragma unroll
  for (int k = 0; k < kN; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[k][j] = 0.0f;
  int turn = 0;
  for (int64_t t = unit; t < p.T; t += gridDim.x * G::kRows) {
    const char* const dyr = static_cast<const char*>(p.dy) + t * p.dy_ld * size;
    const char* const hr = static_cast<const char*>(p.h) + t * p.h_ld * size;
    const char* const dhr = static_cast<const char*>(p.dh) + t * p.dh_ld * size;
    char* const dxr = static_cast<char*>(p.dx) + t * p.dx_ld * size;
    const float r = p.rstd[t];
    Vec<kBF16> a[kN], u[kN], g[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int v = lane + k * G::kLanes;
      if (v >= nvec) continue;
      a[k].load(dyr, v);
      u[k].load(hr, v);
      if (p.dh) g[k].load(dhr, v);
    }
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int v = lane + k * G::kLanes;
      if (v >= nvec) continue;
      float af[8], uf[8], w[8];
      Vec<kWBF16> wv;
      wv.load(p.weight, v);
      wv.get(w);
      a[k].get(af);
      u[k].get(uf);
#pragma unroll
      for (int j = 0; j < 8; ++j) dot += af[j] * w[j] * (uf[j] * r);
    }
    const float mean = G::sum(dot, s_sum[turn]) * inv_d;
    turn ^= 1;  // the next row's slots: this row's may still be read
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int v = lane + k * G::kLanes;
      if (v >= nvec) continue;
      float af[8], uf[8], w[8], o[8];
      Vec<kWBF16> wv;
      wv.load(p.weight, v);
      wv.get(w);
      a[k].get(af);
      u[k].get(uf);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float uj = uf[j] * r;
        acc[k][j] += af[j] * uj;
        o[j] = r * (af[j] * w[j] - uj * mean);
      }
      if (p.dh) {
        float gf[8];
        g[k].get(gf);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += gf[j];
      }
      Vec<kBF16> ov;
      ov.set(o);
      ov.store(dxr, v);
    }
  }
  if (!p.part) return;
  // rows of one workgroup leave one partial sum, added in order
  extern __shared__ float s_part[];
#pragma unroll
  for (int w = 0; w + 1 < G::kRows; ++w) {
    if (G::row() == w) {
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int v = lane + k * G::kLanes;
        if (v >= nvec) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float* const at = s_part + j * G::kLanes * kN + v;
          *at = w == 0 ? acc[k][j] : *at + acc[k][j];
        }
      }
    }
    __syncthreads();
  }
  if (G::row() != G::kRows - 1) return;
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int v = lane + k * G::kLanes;
    if (v >= nvec) continue;
    if (G::kRows > 1)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[k][j] += s_part[j * G::kLanes * kN + v];
    Vec<false> ov;
    ov.set(acc[k]);
    ov.store(p.part + (int64_t)blockIdx.x * p.D, v);
  }
}

// dweight of 32 columns a workgroup: 32 threads of a column take the partial
// sums in turn, then one adds theirs in order.
__global__ __launch_bounds__(1024) void k_rms_dweight(const float* part, int n, int64_t D, float* dw, int accumulate) {
  __shared__ float s[32][33];
  const int l = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + l;
  float sum = 0.0f;
  if (c < D)
#pragma unroll 8
    for (int i = slice; i < n; i += 32) sum += part[i * D + c];
  s[slice][l] = sum;
  __syncthreads();
  if (slice != 0 || c >= D) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) sum += s[i][l];
  dw[c] = accumulate ? dw[c] + sum : sum;
}

template <int kN>
using Int = std::integral_constant<int, kN>;

// Lanes of a row and vectors of a lane for rows of D elements: f(kL, kN).  What
// counts is that no lane idles, that a lane has a few loads on their way and
// that joining a row takes few steps.  2^26 bf16 elements with a residual (537 MB
// moved; their E4M3 form 201 MB) in us, the choice and its neighbours (a group
// of 128 needs 16 lanes):
//   D = 32      4 x 1   96           16 x 1  209
//   D = 64      8 x 1   93           16 x 1  119            4 x 2  107
//   D = 128    16 x 1   95 /  74     64 x 1  224 / 255      8 x 2   98
//   D = 256    16 x 2   96 /  63     32 x 1   97 /  79     64 x 1  126 / 136
//   D = 512    32 x 2   96 /  64     16 x 4  101 /  62     64 x 1   92 /  78
//   D = 1000   64 x 2   98           32 x 4  118           16 x 8  123
//   D = 2048   64 x 4   99 /  61     32 x 8  106 /  65    256 x 1   92 /  82
//   D = 4096  256 x 2   95 /  63    128 x 4   99 /  59    512 x 1   92 /  82
//   D = 8192  256 x 4  100 /  60    512 x 2   96 /  65   1024 x 1   96 /  84
//   D = 16384 512 x 4  101 /  61   1024 x 2  101 /  71    256 x 8  107 /  63
//   D = 32768 1024 x 4 106 /  65    512 x 8  109 /  65
template <class F>
void by_width(int64_t D, F&& f) {
  if (D <= 32) f(Int<4>(), Int<1>());
  else if (D <= 64) f(Int<8>(), Int<1>());
  else if (D <= 128) f(Int<16>(), Int<1>());
  else if (D <= 256) f(Int<16>(), Int<2>());
  else if (D <= 512) f(Int<32>(), Int<2>());
  else if (D <= 1024) f(Int<64>(), Int<2>());
  else if (D <= 2048) f(Int<64>(), Int<4>());
  else if (D <= 4096) f(Int<256>(), Int<2>());
  else if (D <= 8192) f(Int<256>(), Int<4>());
  else if (D <= 16384) f(Int<512>(), Int<4>());
  else f(Int<1024>(), Int<4>());
}

// The same for the gradient, which holds three vectors and a sum for each.  2^26
// elements with dh and dweight (537 MB), the choice and its neighbour: D = 4096
// 256 x 2 104, 128 x 4 115; 8192 512 x 2 106, 256 x 4 118; 16384 1024 x 2 113,
// 512 x 4 125; 32768 1024 x 4 153 (its 128 registers do not hold it all), 512 x
// 8 201 us.
template <class F>
void by_grad_width(int64_t D, F&& f) {
  if (D <= 4096) by_width(D, f);
  else if (D <= 8192) f(Int<512>(), Int<2>());
  else if (D <= 16384) f(Int<1024>(), Int<2>());
  else f(Int<1024>(), Int<4>());
}

// Workgroups that walk the gradient's rows, each with one partial sum of
// dweight: a fixed number, so that a call's sums do not depend on the device.
// Four a CU where several rows share one, two, then one of 1024 threads, which
// no other fits beside (the same 2^26 elements, D = 128: 1024 / 512 workgroups
// 106 / 126 us; 1000: 108 / 108; 2048: 113 / 110; 4096, 512 / 256: 104 / 131;
// 16384: 120 / 113; 32768: 175 / 153).
int grad_blocks(int64_t T, int64_t D) {
  int rows = 1;
  if (D <= 2048) by_width(D, [&](auto l, auto) { rows = Group<decltype(l)::value>::kRows; });
  const int64_t most = D <= 1024 ? 1024 : D <= 8192 ? 512 : 256;
  return (int)std::max<int64_t>(1, std::min<int64_t>((T + rows - 1) / rows, most));
}

bool row_ok(const void* p, int64_t ld, int size) { return aligned16(p) && (ld * size) % 16 == 0; }

}  // namespace
}  // namespace nvq

using namespace nvq;

extern "C" int nvq_rms_norm(const nvq_rms_norm_args* a, void* stream) {
  if (!a || a->struct_size < sizeof(nvq_rms_norm_args)) return NVQ_EINVAL;
  if ((a->dtype != NVQ_F32 && a->dtype != NVQ_BF16) || (a->w_dtype != NVQ_F32 && a->w_dtype != NVQ_BF16)) return NVQ_EINVAL;
  if (!(a->eps >= 0.0) || !(a->eps < 1e300)) return NVQ_EINVAL;
  if (a->T < 0 || a->T > kMaxTokens || a->D < 8 || a->D % 8 != 0 || a->D > kMaxD) return NVQ_ESHAPE;
  if (a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128) return NVQ_EINVAL;
  if (a->y8 && a->group && a->D % a->group != 0) return NVQ_ESHAPE;
  if (a->T != 0 && a->out_amax && !a->y) return NVQ_EINVAL;
  const int size = a->dtype == NVQ_BF16 ? 2 : 4;
  NormParams p;
  p.T = a->T; p.D = a->D;
  p.x_ld = a->x_ld ? a->x_ld : a->D;
  p.res_ld = a->res_ld ? a->res_ld : a->D;
  p.h_ld = a->h_ld ? a->h_ld : a->D;
  p.y_ld = a->y_ld ? a->y_ld : a->D;
  if (p.x_ld < a->D || p.res_ld < a->D || p.h_ld < a->D || p.y_ld < a->D) return NVQ_ESHAPE;
  if (!a->weight) return NVQ_EINVAL;
  if (a->T != 0 && (!a->x || (a->residual && !a->h) || (!a->y && !a->y8) || (a->y8 && !a->y8_scales))) return NVQ_EINVAL;
  if (a->T != 0 && a->residual && a->y == a->h) return NVQ_EINVAL;  // y would take h's place
  if (!row_ok(a->x, p.x_ld, size) || !row_ok(a->residual, p.res_ld, size) || !row_ok(a->h, p.h_ld, size) ||
      !row_ok(a->y, p.y_ld, size) || !aligned16(a->weight) || ((uintptr_t)a->y8 & 7u) || ((uintptr_t)a->y8_scales & 3u) ||
      ((uintptr_t)a->rstd & 3u) || ((uintptr_t)a->out_amax & 3u))
    return NVQ_EALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a->out_amax) {
    hipLaunchKernelGGL(k_zero_word, dim3(1), dim3(1), 0, s, reinterpret_cast<uint32_t*>(a->out_amax));
    if (int rc = last_launch()) return rc;
  }
  if (a->T == 0) return NVQ_OK;
  p.x = a->x; p.res = a->residual; p.weight = a->weight; p.eps = a->eps;
  p.h = a->residual ? a->h : nullptr; p.y = a->y; p.y8 = a->y8; p.scales = a->y8_scales; p.group = a->group;
  p.rstd = a->rstd; p.amax = reinterpret_cast<uint32_t*>(a->out_amax);
  const bool xb = a->dtype == NVQ_BF16, wb = a->w_dtype == NVQ_BF16;
  by_width(a->D, [&](auto w, auto n) {
    constexpr int kL = decltype(w)::value, kN = decltype(n)::value;
    auto pick = [&](auto out) {
      constexpr int kOut = decltype(out)::value;
      return xb ? (wb ? k_rms_norm<true, true, kOut, kL, kN> : k_rms_norm<true, false, kOut, kL, kN>)
                : (wb ? k_rms_norm<false, true, kOut, kL, kN> : k_rms_norm<false, false, kOut, kL, kN>);
    };
    const auto fn = !a->y8 ? pick(std::integral_constant<int, 0>())
                           : a->group ? pick(std::integral_constant<int, 1>()) : pick(std::integral_constant<int, 2>());
    constexpr int64_t rows = Group<kL>::kRows;
    const int64_t groups = (a->T + rows - 1) / rows, gx = std::min<int64_t>(groups, 1 << 21);  // gx * threads < 2^32
    hipLaunchKernelGGL(fn, dim3((unsigned)gx, (unsigned)((groups + gx - 1) / gx)), dim3(Group<kL>::kThreads), 0, s, p);
  });
  return last_launch();
}

extern "C" size_t nvq_rms_norm_backward_workspace_bytes(int64_t T, int64_t D) {
  if (T < 0 || D < 1) return kAlign;
  WsCarve c(nullptr);
  c.take<float>((size_t)grad_blocks(T, D) * D);
  return c.off;
}

extern "C" int nvq_rms_norm_backward(const nvq_rms_norm_grad_args* a, void* stream) {
  if (!a || a->struct_size < sizeof(nvq_rms_norm_grad_args)) return NVQ_EINVAL;
  if ((a->dtype != NVQ_F32 && a->dtype != NVQ_BF16) || (a->w_dtype != NVQ_F32 && a->w_dtype != NVQ_BF16)) return NVQ_EINVAL;
  if (a->T < 0 || a->T > kMaxTokens || a->D < 8 || a->D % 8 != 0 || a->D > kMaxD) return NVQ_ESHAPE;
  const int size = a->dtype == NVQ_BF16 ? 2 : 4;
  NormGradParams p;
  p.T = a->T; p.D = a->D;
  p.dy_ld = a->dy_ld ? a->dy_ld : a->D;
  p.h_ld = a->h_ld ? a->h_ld : a->D;
  p.dh_ld = a->dh_ld ? a->dh_ld : a->D;
  p.dx_ld = a->dx_ld ? a->dx_ld : a->D;
  if (p.dy_ld < a->D || p.h_ld < a->D || p.dh_ld < a->D || p.dx_ld < a->D) return NVQ_ESHAPE;
  if (!a->weight || (a->T != 0 && (!a->dy || !a->h || !a->rstd || !a->dx))) return NVQ_EINVAL;
  if (!row_ok(a->dy, p.dy_ld, size) || !row_ok(a->h, p.h_ld, size) || !row_ok(a->dh, p.dh_ld, size) ||
      !row_ok(a->dx, p.dx_ld, size) || !aligned16(a->weight) || ((uintptr_t)a->rstd & 3u) || ((uintptr_t)a->dweight & 3u))
    return NVQ_EALIGN;
  if (a->dweight) {
    if (!a->ws || a->ws_bytes < nvq_rms_norm_backward_workspace_bytes(a->T, a->D)) return NVQ_EWORKSPACE;
    if (!aligned256(a->ws)) return NVQ_EALIGN;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int blocks = grad_blocks(a->T, a->D);
  WsCarve c(a->ws);
  p.part = a->dweight ? c.take<float>((size_t)blocks * a->D) : nullptr;
  p.dy = a->dy; p.h = a->h; p.weight = a->weight; p.rstd = a->rstd; p.dh = a->dh; p.dx = a->dx;
  if (a->T != 0) {
    const bool xb = a->dtype == NVQ_BF16, wb = a->w_dtype == NVQ_BF16;
    by_grad_width(a->D, [&](auto w, auto n) {
      constexpr int kL = decltype(w)::value, kN = decltype(n)::value;
      auto fn = xb ? (wb ? k_rms_grad<true, true, kL, kN> : k_rms_grad<true, false, kL, kN>)
                   : (wb ? k_rms_grad<false, true, kL, kN> : k_rms_grad<false, false, kL, kN>);
      const size_t lds = Group<kL>::kRows > 1 && p.part ? sizeof(float) * 8 * Group<kL>::kLanes * kN : 0;
      hipLaunchKernelGGL(fn, dim3(blocks), dim3(Group<kL>::kThreads), lds, s, p);
    });
    if (int rc = last_launch()) return rc;
  }
  if (!a->dweight) return NVQ_OK;
  hipLaunchKernelGGL(k_rms_dweight, dim3((unsigned)((a->D + 31) / 32)), dim3(1024), 0, s, p.part,
                     a->T ? blocks : 0, a->D, a->dweight, a->accumulate);
  return last_launch();
}
