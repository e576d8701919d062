// Linear cross entropy: softmax cross entropy of x w^T without keeping the
// logits, and its gradient (gfx950).
//
//   z[t, v] = scale x[t] . w[v]
//   lse[t]  = ln sum_v exp z[t, v],  loss[t] = lse[t] - z[t, y_t]
//   c[t, v] = exp(z[t, v] - lse[t]) - [v = y_t]
//   dx[t]   = scale dloss_t sum_v c[t, v] w[v]
//   dw[v]   = scale sum_t c[t, v] dloss_t x[t]
//
// Forward: every 256 x 256 tile of logits leaves a maximum and a sum of
// exponentials per token, which one pass joins.  Gradient: the tokens that
// count (a valid target, dloss not 0) are gathered into a dense copy first, so
// padded tokens cost nothing and nothing they hold (NaN included) reaches the
// sums.  A token's weight dloss / g is split into m 2^e, 1 <= m < 2: m goes into
// c, 2^e with the sign into the token's row of x (exactly) and of dx.  The
// vocabulary then goes by in pieces: logits again, m c rounded to bf16 (2^-8
// relative at most, the only rounding to fewer bits on the way to dx and dw; the
// entries of improbable targets, which carry most of the gradient, round to -1
// with hardly any error where m is 1, as in a mean loss; where weights differ,
// what the rounding took from a target's own terms is added again), and the two
// products of m c with w and with 2^e x.  dx is summed in fp32 over the pieces.
//
// Bound by the matrix cores' power: 8192 tokens, 65536 words of 4096 (four
// products of 4.4 TFLOP) take 3.3 + 10.5 ms (3.4 + 10.9 on another card), 1.27 PFLOP/s, the
// tiles of 256 alone 1.33 (forward), 1.23 (c), 1.31 (dx) and 1.29 (dw).  Few
// tokens are bound by w's bytes: one token, 131072 words of 7168, 309 us (6.1 TB/s).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "nvq.h"
#include "nvq_device.h"
#include "nvq_gemm_bf16.h"
#include "nvq_internal.h"

namespace nvq {
namespace {

using gemm::f32x16;

constexpr int kTile = 256;  // tiles are counted in this size, whatever takes them

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What the gradient's kernels read of the tokens that count.
struct Live {
  int32_t* count;   // [1]
  float* g;         // [1] max |dloss|; dloss / g = m 2^e, 1 <= m < 2, and a sign
  int32_t* row;     // [T] token of live row i
  int32_t* pos;     // [T] live row of a token, or -1
  uint16_t* x;      // [Tp, Dx] their states, zeros behind the last and past D
  uint16_t* xr;     // [Tp, Dx] the same times 2^e and the sign
  float* m;         // [Tp]
  float* l2;        // [Tp] lse in bits, less log2 m
  int32_t* y;       // [Tp]
  float* cy;        // [T] m c of the target
  int32_t* uneven;  // [1] whether any m may differ from 1
};

struct CeParams {
  int64_t T, D, V;
  const uint16_t* x;
  int64_t x_ld;
  const uint16_t* w;
  int64_t w_ld;
  const int32_t* targets;
  float scale;
  float* loss;
  float* lse;
  const float* dloss;
  uint16_t* dx;
  int64_t dx_ld;
  void* dw;
  int64_t dw_ld;
  uint32_t* status;
  // forward
  float2* part;     // [vocabulary tiles, T] (maximum in bits, sum)
  float* at;        // [T] the target's logit in bits
  // gradient
  Live live;
  int64_t Dx;       // row length of live.x
  uint16_t* c;      // [Tp, Vp] of the piece
  int64_t Vp;
  float* slab;      // [slices, Tp, D]
  int64_t Tp;
  int slices;
  int64_t v0, v1;   // the piece
  int first;        // the first piece of the call
  // the tiles that a launch takes: these of the order of pick(), whole or as quarters
  int tile0, tile1;
};

// Runs a workgroup's tile.  XCD b % 8 takes a contiguous range of an order that
// walks groups of 8 tiles along m first, so that what one XCD runs at a time
// shares panels in its L2.  A launch has the tiles tile0 .. tile1 - 1 of the
// order (of those that there are: some sizes are known on the device only), as
// tiles of 256 (kF == 4) or each as four of 128 (kF == 2).  panels(m0, n0, A, B)
// describes a tile's operands (false: it holds nothing), store(m0, n0, acc)
// takes its results; lds is free again by then.  With slices of the contraction
// the order goes through all tiles of one after the other, so that an XCD keeps
// to its own part of both operands.
// One workgroup a tile: persistent workgroups that sent the next tile's first
// stages on their way before they stored took 3 to 7 % more time (loss and
// gradient of 8192 tokens, 65536 words of 4096: 14.16 ms against 13.71; 1023,
// 50001 of 1000: 542 us against 505): tiles then wait for their own workgroup,
// where here any free CU takes them.
template <int kF, bool kRowsA, bool kRowsB, bool kTurn, class Panels, class Store>
__device__ __forceinline__ void run_tile(const CeParams& p, int64_t rows_m, int64_t rows_n, char* lds, Panels&& panels,
                                         Store&& store, int slices = 1, int* slice = nullptr) {
  constexpr int kGroup = 8, kSub = kF == 4 ? 1 : 4;
  const int nm = (int)((rows_m + kTile - 1) / kTile), nn = (int)((rows_n + kTile - 1) / kTile);
  const int tiles = max(0, min(p.tile1, nm * nn) - p.tile0) * kSub, total = tiles * slices, per = (total + 7) / 8;
  const int slot = blockIdx.x >> 3, b = (blockIdx.x & 7) * per + slot;
  if (slot >= per || b >= total) return;
  if (slice) *slice = b / tiles;
  const int in = slices > 1 ? b % tiles : b, t = p.tile0 + in / kSub, sub = in % kSub;
  const int span = kGroup * nn, grp = t / span, rem = t - grp * span;
  const int rows = min(kGroup, nm - grp * kGroup);
  const int64_t n0 = (int64_t)(rem / rows) * kTile + 128 * (sub >> 1);
  const int64_t m0 = (int64_t)(grp * kGroup + rem % rows) * kTile + 128 * (sub & 1);
  gemm::Panel A, B;
  if (!panels(m0, n0, A, B)) return;
  f32x16 acc[kF][kF];
  {
    gemm::Product<kF, kRowsA, kRowsB, kTurn> product(lds);
    product.begin(A, B);
    product.run(acc);
  }
  store(m0, n0, acc);
}
inline unsigned grid_of(int64_t tiles) { return (unsigned)((tiles + 7) / 8 * 8); }

// acc element v of block i -> row of the wave's 32 kF, less 4 h
__device__ __forceinline__ constexpr int row_of(int i, int v) { return 32 * i + 8 * (v >> 2) + (v & 3); }

// This lane's number, as a value that the compiler cannot use earlier: the
// addresses that a tile's results need are computed where the registers are
// free, instead of being kept (or spilled) during the products.
__device__ __forceinline__ int lane_here() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

constexpr int kPart = 128;  // words of a partial result

// Joins (maximum, sum of 2^(value - maximum)) with another such pair.
__device__ __forceinline__ void join(float& m, float& sum, float2 q) {
  const float top = __builtin_fmaxf(m, q.x), ref = top == -INFINITY ? 0.0f : top;
  sum = sum * __builtin_amdgcn_exp2f(m - ref) + q.y * __builtin_amdgcn_exp2f(q.x - ref);
  m = top;
}

// ---------------------------------------------------------------- forward --
template <int kF, bool kTurn>
__global__ __launch_bounds__(gemm::kThreads, kF == 4 ? 1 : 2) void k_ce_forward(CeParams p) {
  constexpr int kEdge = 64 * kF, kWave = 32 * kF;
  __shared__ __attribute__((aligned(16))) char lds[gemm::Shape<kF>::kLdsBytes];
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float k2 = p.scale * kLog2e;
  run_tile<kF, false, false, kTurn>(
      p, p.V, p.T, lds,
      [&](int64_t v0, int64_t t0, gemm::Panel& A, gemm::Panel& B) -> bool {
        if (v0 >= p.V || t0 >= p.T) return false;  // a quarter outside
        A = {p.w + v0 * p.w_ld, (uint32_t)p.w_ld, (int)min<int64_t>(kEdge, p.V - v0), p.D};
        B = {p.x + t0 * p.x_ld, (uint32_t)p.x_ld, (int)min<int64_t>(kEdge, p.T - t0), p.D};
        return true;
      },
      [&](int64_t v0, int64_t t0, f32x16 (&acc)[kF][kF]) {
        const int lane = lane_here(), l32 = lane & 31, h = lane >> 5;
        const int64_t vw = v0 + kWave * (wave & 1);
        const int have = (int)min<int64_t>(kWave, max<int64_t>(0, p.V - vw));  // words of this wave's rows
        float2* const s_half = reinterpret_cast<float2*>(lds);  // kF == 2: [2][128]
#pragma unroll
        for (int j = 0; j < kF; ++j) {
          const int64_t t = t0 + kWave * (wave >> 1) + 32 * j + l32;
          float z[kF][16];
#pragma unroll
          for (int i = 0; i < kF; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) z[i][v] = acc[i][j][v] * k2;
          const int y = t < p.T ? (int)min<int64_t>(p.targets[t] - vw, (int64_t)kWave) : -1;
          if (__any(y >= 0 && y < have)) {
            float hit = 0.0f;
#pragma unroll
            for (int i = 0; i < kF; ++i)
#pragma unroll
              for (int v = 0; v < 16; ++v) hit = row_of(i, v) == y - 4 * h ? z[i][v] : hit;
            if (y >= 0 && y < have && ((y >> 2) & 1) == h) p.at[t] = hit;
          }
          if (have < kWave) {
#pragma unroll
            for (int i = 0; i < kF; ++i)
#pragma unroll
              for (int v = 0; v < 16; ++v) z[i][v] = row_of(i, v) < have - 4 * h ? z[i][v] : -INFINITY;
          }
          float m = -INFINITY;
#pragma unroll
          for (int i = 0; i < kF; ++i)
#pragma unroll
            for (int v = 0; v < 16; v += 2) m = __builtin_fmaxf(__builtin_fmaxf(m, z[i][v]), z[i][v + 1]);
          m = __builtin_fmaxf(m, __shfl_xor(m, 32, 64));
          const float ref = m == -INFINITY ? 0.0f : m;
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
          for (int i = 0; i < kF; ++i)
#pragma unroll
            for (int v = 0; v < 16; v += 2) {
              s0 += __builtin_amdgcn_exp2f(z[i][v] - ref);
              s1 += __builtin_amdgcn_exp2f(z[i][v + 1] - ref);
            }
          float s = s0 + s1;
          s += __shfl_xor(s, 32, 64);
          if (kF == 2) {
            if (h == 0) s_half[128 * (wave & 1) + kWave * (wave >> 1) + 32 * j + l32] = make_float2(m, s);
          } else if (h == 0 && t < p.T && have > 0) {
            p.part[(vw / kPart) * p.T + t] = make_float2(m, s);
          }
          __builtin_amdgcn_sched_barrier(0);  // one block's values in registers at a time
        }
        if (kF == 4) return;
        __syncthreads();
        const int64_t t = t0 + threadIdx.x;
        if (threadIdx.x < 128 && t < p.T) {
          float2 a = s_half[threadIdx.x];
          join(a.x, a.y, s_half[128 + threadIdx.x]);
          p.part[(v0 / kPart) * p.T + t] = a;
        }
      });
}

// Few tokens: every row of w is read once, which is all the time there is (64
// tokens at a time where there are more).  A workgroup takes 64 words at a time;
// its four waves share the contraction (wave q the 64-element steps q, q + 4,
// ..), so together they read 512 contiguous bytes of each row.  Lane (l16, g) of v_mfma_f32_16x16x32_bf16 holds
// the 32 bytes 32 g .. of row l16 of a step's 128 as two operands; x is held in
// the same order, so the contraction is only permuted.  The next step's rows of
// w (the next 64 words', at the end) are on their way while this one is
// multiplied; x comes from the L2.  The waves' sums meet in LDS, where each thread has one token and
// every n-th word, and keeps that token's running maximum and sum.
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 tokens, 65536 words of 4096: 104 us, 5.2 TB/s of w.
constexpr int kFew = 64;  // tokens of a workgroup at most

template <int kN>  // 16-token operands
__global__ __launch_bounds__(256, 2) void k_ce_few(CeParams p) {
  constexpr int kTok = 16 * kN, kPitch = kTok + 4, kPer = 256 / kTok;
  __shared__ float red[4 * 64 * kPitch];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = 0u;
  const int64_t t0 = (int64_t)blockIdx.y * kTok, T = min<int64_t>(kTok, p.T - t0);  // this workgroup's tokens
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = (int)((p.D + 255) / 256);  // steps of 64 words
  const uint32_t w_row = (uint32_t)(p.w_ld * 2), x_row = (uint32_t)(p.x_ld * 2);
  const uint32_t w_off = l16 * w_row + 32 * g, x_off = l16 * x_row + 32 * g;
  struct Set {
    u32x4 w[4][2];
  } set[2];
  u32x4 x[kN][2];
  // descriptors end with the last row's last element; a lane whose 8 elements
  // lie behind its own row's is sent past that end
  auto fetch = [&](const uint16_t* base, uint32_t off, uint32_t row, int rows, int step, auto&& to, auto count) {
    const int k = 64 * (4 * step + wave), left = (int)p.D - k;
    const auto d = __builtin_amdgcn_make_buffer_rsrc((void*)(base + k), 0, left > 0 ? (int)((rows - 1) * row) + 2 * left : 0, 0x00020000);
    uint32_t out[2] = {0, 0};
    if (left < 64)
#pragma unroll
      for (int u = 0; u < 2; ++u) out[u] = 16 * g + 8 * u < left ? 0u : 0x80000000u;
#pragma unroll
    for (int f = 0; f < decltype(count)::value; ++f)
#pragma unroll
      for (int u = 0; u < 2; ++u) to[f][u] = __builtin_amdgcn_raw_buffer_load_b128(d, (off + 16 * f * row + 16 * u) | out[u], 0, 0);
  };
  auto load_w = [&](Set& s, int64_t v0, int step) {
    fetch(p.w + v0 * p.w_ld, w_off, w_row, (int)min<int64_t>(64, p.V - v0), step, s.w, std::integral_constant<int, 4>());
  };
  f32x4 acc[4][kN];
  auto clear = [&] {
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int c = 0; c < kN; ++c) acc[f][c] = 0.0f;
  };
  clear();
  const int tok = threadIdx.x % kTok, part = threadIdx.x / kTok;
  const int64_t y = tok < T ? p.targets[t0 + tok] : -1;
  const float k2 = p.scale * kLog2e;
  float m = -INFINITY, sum = 0.0f;
  int64_t v0 = (int64_t)blockIdx.x * 64;  // words and step of the set in hand
  int at = 0;
  // multiplies `now`, loads what follows it; false behind the last step
  auto step = [&](Set& now, Set& next) -> bool {
    const bool last = at == n - 1;
    const int64_t nv = last ? v0 + 64 * (int64_t)gridDim.x : v0;
    const bool more = nv < p.V;
    fetch(p.x + t0 * p.x_ld, x_off, x_row, (int)T, at, x, std::integral_constant<int, kN>());
    if (more) load_w(next, nv, last ? 0 : at + 1);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int c = 0; c < kN; ++c)
          acc[f][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(gemm::bf16x8, now.w[f][u]),
                                                              __builtin_bit_cast(gemm::bf16x8, x[c][u]), acc[f][c], 0, 0, 0);
    if (!last) {
      ++at;
      return true;
    }
    // the words of this tile are done: acc[f][c][v] is word 16 f + 4 g + v, token 16 c + l16
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int c = 0; c < kN; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[(64 * wave + 16 * f + 4 * g + v) * kPitch + 16 * c + l16] = acc[f][c][v];
    clear();
    __syncthreads();
    float z[64 / kPer];
    float top = m;
#pragma unroll
    for (int i = 0; i < 64 / kPer; ++i) {
      const int v = part + i * kPer;
      const float* const q = red + v * kPitch + tok;
      const float d = (q[0] + q[64 * kPitch]) + (q[128 * kPitch] + q[192 * kPitch]);
      z[i] = v0 + v < p.V ? d * k2 : -INFINITY;
      if (v0 + v == y && y < p.V) p.at[t0 + tok] = z[i];
      top = __builtin_fmaxf(top, z[i]);
    }
    const float ref = top == -INFINITY ? 0.0f : top;
    sum *= __builtin_amdgcn_exp2f(m - ref);
#pragma unroll
    for (int i = 0; i < 64 / kPer; ++i) sum += __builtin_amdgcn_exp2f(z[i] - ref);
    m = top;
    v0 = nv;
    at = 0;
    __syncthreads();
    return more;
  };
  load_w(set[0], v0, 0);
  while (step(set[0], set[1]) && step(set[1], set[0])) {
  }
  // the kPer threads of a token, in order
  float2* const s = reinterpret_cast<float2*>(red);
  s[part * kTok + tok] = make_float2(m, sum);
  __syncthreads();
  if (part != 0 || tok >= T) return;
  for (int i = 1; i < kPer; ++i) join(m, sum, s[i * kTok + tok]);
  p.part[(int64_t)blockIdx.x * p.T + t0 + tok] = make_float2(m, sum);
}

// lse and loss of 8 tokens a workgroup: 128 threads of a token take the partial
// results in turn, 8 join 16 of those each, one the 8.
__global__ __launch_bounds__(1024) void k_ce_join(CeParams p, int parts) {
  __shared__ float2 s[128][9];
  const int l = threadIdx.x & 7, part = threadIdx.x >> 3;
  const int64_t t = (int64_t)blockIdx.x * 8 + l;
  float m = -INFINITY, sum = 0.0f;
  if (t < p.T)
#pragma unroll 4
    for (int i = part; i < parts; i += 128) join(m, sum, p.part[(int64_t)i * p.T + t]);
  s[part][l] = make_float2(m, sum);
  __syncthreads();
  if (part < 8) {
#pragma unroll
    for (int i = 1; i < 16; ++i) join(m, sum, s[8 * i + part][l]);
  }
  __syncthreads();
  if (part < 8) s[part][l] = make_float2(m, sum);
  __syncthreads();
  if (part != 0 || t >= p.T) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) join(m, sum, s[i][l]);
  // The loss is the target's distance from the maximum, in bits, and what the sum
  // adds to it, never the difference of two large numbers: a token whose target
  // leads has the loss that the others leave it, and none is negative (tokens with
  // logits of 2000 were off by 1.2e-4 as lse - logit).
  const float rest = logf(sum);
  if (p.lse) p.lse[t] = m * kLn2 + rest;
  const int64_t y = p.targets[t];
  if (y >= p.V) atomicOr(p.status, (uint32_t)NVQ_STATUS_BAD_TARGET);
  if (p.loss) p.loss[t] = y >= 0 && y < p.V ? (m - p.at[t]) * kLn2 + rest : 0.0f;
}

// --------------------------------------------------------------- gradient --
// Finds the tokens that count, in order, the largest |dloss|, and whether the
// weights are more than powers of two apart.
__global__ __launch_bounds__(1024) void k_ce_live(CeParams p) {
  __shared__ int s_n[16];
  __shared__ uint32_t s_g[16], s_bad[16], s_ones[16], s_zeros[16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int base = 0;
  uint32_t top = 0, bad = 0;
  uint32_t ones = 0, zeros = 0;  // mantissa bits that some weight has set, clear
  for (int64_t t0 = 0; t0 < p.T; t0 += 1024) {
    const int64_t t = t0 + threadIdx.x;
    bool live = false;
    if (t < p.T) {
      const int64_t y = p.targets[t];
      const float d = p.dloss ? p.dloss[t] : 1.0f;
      bad |= y >= p.V;
      live = y >= 0 && y < p.V && d != 0.0f;  // a NaN counts
      const uint32_t a = __float_as_uint(d) & 0x7FFFFFFFu;
      if (live && a < 0x7F800000u) top = max(top, a);
      if (live) {
        ones |= a < 0x800000u ? ~0u : a & 0x7FFFFFu;  // numbers below the normal ones count as uneven
        zeros |= ~a & 0x7FFFFFu;
      }
    }
    const uint64_t mask = __ballot(live);
    if (lane == 0) s_n[wave] = __popcll(mask);
    __syncthreads();
    int at = base + __popcll(mask & ((1ull << lane) - 1ull));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      at += i < wave ? s_n[i] : 0;
      base += s_n[i];
    }
    if (t < p.T) p.live.pos[t] = live ? at : -1;
    if (live) p.live.row[at] = (int32_t)t;
    __syncthreads();
  }
  top = wave_max_u32(top);
  bad = wave_or_u32(bad);
  ones = wave_or_u32(ones);
  zeros = wave_or_u32(zeros);
  if (lane == 0) {
    s_g[wave] = top;
    s_bad[wave] = bad;
    s_ones[wave] = ones;
    s_zeros[wave] = zeros;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < 16; ++i) {
    top = max(top, s_g[i]);
    bad |= s_bad[i];
    ones |= s_ones[i];
    zeros |= s_zeros[i];
  }
  *p.live.count = base;
  *p.live.uneven = (ones & zeros) != 0;  // r is a power of two where all mantissas are alike
  *p.live.g = top ? __uint_as_float(top) : 1.0f;  // only non-finite weights: they stand for themselves
  *p.status = bad ? (uint32_t)NVQ_STATUS_BAD_TARGET : 0u;
}

// The dense copies: one workgroup a row, up to the last row's tile.
__global__ __launch_bounds__(256) void k_ce_gather(CeParams p) {
  const int64_t i = blockIdx.x;
  const int64_t n = *p.live.count;
  if (i >= (n + kTile - 1) / kTile * kTile) return;
  const bool live = i < n;
  const int64_t t = live ? p.live.row[i] : 0;
  uint4* const to = reinterpret_cast<uint4*>(p.live.x + i * p.Dx);
  const uint4* const from = reinterpret_cast<const uint4*>(p.x + t * p.x_ld);
  uint4* const tor = reinterpret_cast<uint4*>(p.live.xr + i * p.Dx);
  const float r = live ? (p.dloss ? p.dloss[t] : 1.0f) / *p.live.g : 0.0f;
  // a weight that is no number, or vanishes beside g, stands for itself
  const bool split = __builtin_isfinite(r) && r != 0.0f;
  const float m = split ? 2.0f * __builtin_amdgcn_frexp_mantf(fabsf(r)) : 1.0f;
  const float e = split ? copysignf(ldexpf(1.0f, __builtin_amdgcn_frexp_expf(r) - 1), r) : r;
  for (int k = threadIdx.x; k < (int)(p.Dx / 8); k += 256) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (live && 8 * k < p.D) q = from[k];
    to[k] = q;
    auto times = [&](uint32_t w) { return pack_bf16(bf16_lo(w) * e, bf16_hi(w) * e); };
    tor[k] = make_uint4(times(q.x), times(q.y), times(q.z), times(q.w));
  }
  if (threadIdx.x == 0) {
    p.live.m[i] = m;
    p.live.l2[i] = (live ? p.lse[t] : 0.0f) * kLog2e - (m == 1.0f ? 0.0f : log2f(m));
    p.live.y[i] = live ? p.targets[t] : -1;
  }
}

// Stores a wave's 32 kF (memory rows, along l32) x 32 kF (contiguous) block as
// bf16 rows, 32 rows at a time through 2 kF KB of LDS of its own: 8-byte pieces
// in (the four values v % 4 of a lane are neighbours), 16-byte pieces out.
// Chunk c of row n lies in slot c ^ (n mod the chunks of a row).  f(j, z) turns
// the accumulators of 32 rows into the values to store.
template <int kF, class F, class G>
__device__ __forceinline__ void store_block(char* region, f32x16 (&acc)[kF][kF], F&& f, G&& put) {
  constexpr int kChunks = 4 * kF, kRow = 64 * kF, kAtOnce = 64 / kChunks;
  const int lane = lane_here(), l32 = lane & 31, h = lane >> 5;
#pragma unroll
  for (int j = 0; j < kF; ++j) {
    float z[kF][16];
#pragma unroll
    for (int i = 0; i < kF; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) z[i][v] = acc[i][j][v];
    f(j, z);
#pragma unroll
    for (int i = 0; i < kF; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint2*>(region + l32 * kRow + 16 * ((4 * i + q) ^ (l32 % kChunks)) + 8 * h) =
            make_uint2(pack_bf16(z[i][4 * q], z[i][4 * q + 1]), pack_bf16(z[i][4 * q + 2], z[i][4 * q + 3]));
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS writes are done
    __builtin_amdgcn_wave_barrier();
    uint4 out[2 * kF];
#pragma unroll
    for (int m = 0; m < 2 * kF; ++m) {
      const int n = kAtOnce * m + lane / kChunks, c = lane % kChunks;
      out[m] = *reinterpret_cast<const uint4*>(region + n * kRow + 16 * (c ^ (n % kChunks)));
    }
#pragma unroll
    for (int m = 0; m < 2 * kF; ++m) put(32 * j + kAtOnce * m + lane / kChunks, lane % kChunks, out[m]);
    __builtin_amdgcn_sched_barrier(0);  // one block's values in registers at a time
  }
}

// m c of the piece, tile by tile: [live rows, Vp] bf16, zeros past V (rows behind
// the last hold anything).  8192 x 32768 out of 4096: 1.77 ms, 1.24 PFLOP/s.
template <int kF, bool kTurn>
__global__ __launch_bounds__(gemm::kThreads, kF == 4 ? 1 : 2) void k_ce_coef(CeParams p) {
  constexpr int kEdge = 64 * kF, kWave = 32 * kF;
  __shared__ __attribute__((aligned(16))) char lds[gemm::Shape<kF>::kLdsBytes];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float k2 = p.scale * kLog2e;
  const int64_t n = *p.live.count;
  run_tile<kF, false, false, kTurn>(
      p, p.v1 - p.v0, n, lds,
      [&](int64_t vt, int64_t t0, gemm::Panel& A, gemm::Panel& B) -> bool {
        if (t0 >= n) return false;  // a quarter behind the last row: nothing that counts comes of those
        // a quarter past V has no rows of w: one that counts as zeros (below)
        const int64_t v0 = p.v0 + vt;
        A = {p.w + min<int64_t>(v0, p.V - 1) * p.w_ld, (uint32_t)p.w_ld, (int)max<int64_t>(1, min<int64_t>(kEdge, p.V - v0)), p.D};
        B = {p.live.x + t0 * p.Dx, (uint32_t)p.Dx, kEdge, p.D};
        return true;
      },
      [&](int64_t vt, int64_t t0, f32x16 (&acc)[kF][kF]) {
        const int lane = lane_here(), l32 = lane & 31, h = lane >> 5;
        const int64_t vw = p.v0 + vt + kWave * (wave & 1), tw = t0 + kWave * (wave >> 1);
        const int have = (int)min<int64_t>(kWave, max<int64_t>(0, p.V - vw));
        uint16_t* const out = p.c + tw * p.Vp + (vt + kWave * (wave & 1));
        store_block<kF>(
            lds + 2048 * kF * wave, acc,
            [&](int j, float (&z)[kF][16]) {
              const float l2 = p.live.l2[tw + 32 * j + l32];
              const int y = (int)min<int64_t>(p.live.y[tw + 32 * j + l32] - vw, (int64_t)kWave);
#pragma unroll
              for (int i = 0; i < kF; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v) z[i][v] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[i][v], k2, -l2));
              if (__any(y >= 0 && y < kWave)) {
                const float m = p.live.m[tw + 32 * j + l32];
                float hit = 0.0f;
#pragma unroll
                for (int i = 0; i < kF; ++i)
#pragma unroll
                  for (int v = 0; v < 16; ++v)
                    if (row_of(i, v) == y - 4 * h) hit = z[i][v] -= m;
                if (y >= 0 && y < kWave && ((y >> 2) & 1) == h) p.live.cy[tw + 32 * j + l32] = hit;
              }
              if (have < kWave) {
#pragma unroll
                for (int i = 0; i < kF; ++i)
#pragma unroll
                  for (int v = 0; v < 16; ++v) z[i][v] = row_of(i, v) < have - 4 * h ? z[i][v] : 0.0f;
              }
            },
            [&](int n, int c, uint4 q) { *reinterpret_cast<uint4*>(out + n * p.Vp + 8 * c) = q; });
      });
}

// One slice of the piece's contribution to dx, in fp32 (8192 x 4096 out of 32768
// words: 1.67 ms, 1.32 PFLOP/s).
__global__ __launch_bounds__(gemm::kThreads, 1) void k_ce_dx(CeParams p) {
  __shared__ __attribute__((aligned(16))) char lds[gemm::Shape<4>::kLdsBytes];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int slice = 0;
  const int64_t words = p.v1 - p.v0, steps = (words + gemm::kStep - 1) / gemm::kStep, per = (steps + p.slices - 1) / p.slices;
  const int64_t n = *p.live.count;
  run_tile<4, false, true, false>(
      p, n, p.D, lds,
      [&](int64_t t0, int64_t d0, gemm::Panel& A, gemm::Panel& B) -> bool {
        const int64_t a = min<int64_t>(slice * per * gemm::kStep, words), b = min<int64_t>(a + per * gemm::kStep, words);
        A = {p.c + t0 * p.Vp + a, (uint32_t)p.Vp, kTile, b - a};
        B = {p.w + (p.v0 + a) * p.w_ld + d0, (uint32_t)p.w_ld, (int)min<int64_t>(kTile, p.D - d0), b - a};
        return true;
      },
      [&](int64_t t0, int64_t d0, f32x16 (&acc)[4][4]) {
        const int lane = lane_here(), l32 = lane & 31, h = lane >> 5;
        const int64_t d = d0 + 128 * (wave >> 1) + l32;
        float* const out = p.slab + ((int64_t)slice * p.Tp + t0 + 128 * (wave & 1) + 4 * h) * p.D + d;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (d + 32 * j >= p.D) continue;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (t0 + 128 * (wave & 1) + 32 * i >= n) continue;  // nobody reads rows behind the last (of 32)
            float* const o = out + (int64_t)(32 * i) * p.D + 32 * j;
            if (p.first) {
#pragma unroll
              for (int v = 0; v < 16; ++v) o[row_of(0, v) * p.D] = acc[i][j][v];
            } else {
              float old[16];
#pragma unroll
              for (int v = 0; v < 16; ++v) old[v] = o[row_of(0, v) * p.D];
#pragma unroll
              for (int v = 0; v < 16; ++v) o[row_of(0, v) * p.D] = old[v] + acc[i][j][v];
            }
          }
        }
      },
      p.slices, &slice);
}

// What rounding to bf16 takes from a value (exactly).
__device__ __forceinline__ float lost_of(float f) { return f - bf16_lo(pack_bf16(f, 0.0f)); }

// dx of every token: its slices in order, zero for a token that does not count.
// kSplit: a token's 256 columns take four waves, each a quarter of the slices
// (many slices stand for few tokens; gradient of 20 tokens, 100000 words of 64:
// 69 us instead of 76); else a wave takes 256 columns.  Bound by its reads (2048
// tokens of 2048, four slices: 21 us, 3.6 TB/s).
template <bool kSplit>
__global__ __launch_bounds__(256) void k_ce_dx_join(CeParams p) {
  __shared__ float4 s_sum[4][64];
  const int64_t t = blockIdx.x;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t d = 4 * lane + 256 * (kSplit ? (int64_t)blockIdx.y : 4 * (int64_t)blockIdx.y + wave);
  const int32_t i = p.live.pos[t];
  const int per = (p.slices + 3) / 4, k0 = kSplit ? min(p.slices, wave * per) : 0, k1 = kSplit ? min(p.slices, k0 + per) : p.slices;
  float4 o = make_float4(0, 0, 0, 0);
  if (i >= 0 && d < p.D) {
    const float* const from = p.slab + (int64_t)i * p.D + d;
#pragma unroll 8
    for (int k = k0; k < k1; ++k) {
      const float4 q = *reinterpret_cast<const float4*>(from + (int64_t)k * p.Tp * p.D);
      o = make_float4(o.x + q.x, o.y + q.y, o.z + q.z, o.w + q.w);
    }
  }
  if (kSplit) {
    s_sum[wave][lane] = o;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float4 q = s_sum[w][lane];
      o = make_float4(o.x + q.x, o.y + q.y, o.z + q.z, o.w + q.w);
    }
  }
  if (d >= p.D) return;
  if (i >= 0 && *p.live.uneven) {  // what the target's own m c lost, as add_targets() gives it to dw
    const float lost = lost_of(p.live.cy[i]);
    const uint2 w = *reinterpret_cast<const uint2*>(p.w + (int64_t)p.live.y[i] * p.w_ld + d);
    o = make_float4(__builtin_fmaf(lost, bf16_lo(w.x), o.x), __builtin_fmaf(lost, bf16_hi(w.x), o.y),
                    __builtin_fmaf(lost, bf16_lo(w.y), o.z), __builtin_fmaf(lost, bf16_hi(w.y), o.w));
  }
  const float s = i < 0 ? 0.0f : p.scale * ((p.dloss ? p.dloss[t] : 1.0f) / p.live.m[i]);
  *reinterpret_cast<uint2*>(p.dx + t * p.dx_ld + d) =
      i < 0 ? make_uint2(0, 0) : make_uint2(pack_bf16(o.x * s, o.y * s), pack_bf16(o.z * s, o.w * s));
}

// What the rounding of m c took from a target's own term of dw, added to a tile's
// sums: (m cy - bf16(m cy)) 2^e x as products of bf16 values (what the rounding of
// the first factor takes is 2^-17 of the term), each in a slot of the contraction
// of its own that only the target's word has a factor for.  That term is most of a
// word's gradient, and dx gets back its own in k_ce_dx_join; equal weights skip
// both.  1023 tokens, 50001 words of 1000, weighted: relative error of dw 2.37e-3
// without this, 1.65e-3 with it, all of it dw's own rounding; of dx 2.37e-3 and
// 1.66e-3; loss and gradient 496 and 502 us.  (A weight rounded into the rows of x
// instead left words without a target at 2.30e-3 in fp32; as it is 1.63e-3, one
// rounding of m c.)
// The tokens of a tile's words are searched for each tile: n / 256 loads a
// thread, where the products of n tokens took n / 64 stages of 2048 cycles.  Many
// tokens of few words take several turns; tokens are added in their order.  16
// tokens are one product of the contraction's smallest length, so few words cost
// most (loss and gradient of 8192 tokens, 5000 words of 1024: 424 us with equal
// weights, 449 with others; 1000 words: 210 and 271).
template <int kF>
__device__ __forceinline__ void add_targets(const CeParams& p, char* lds, int n, int64_t v0, int64_t d0, f32x16 (&acc)[kF][kF]) {
  constexpr int kWave = 32 * kF, kU = 2 * kF, kCap = 256 * kF;  // kCap: tokens of a wave's words that one wave finds in a turn
  struct Found {
    uint32_t key;  // token and word
    float lost;
  };
  const int lane = lane_here(), l32 = lane & 31, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int* const count = reinterpret_cast<int*>(lds);         // [2][4]
  int* const more = count + 8;                            // [4]
  Found* const list = reinterpret_cast<Found*>(more + 4);  // [2][4][kCap]
  const int per = ((n + 3) / 4 + 63) / 64 * 64, end = min(n, (wave + 1) * per), half = wave >> 1;
  const int64_t d = d0 + kWave * (wave & 1) + l32;
  for (int at = wave * per;;) {
    int have[2] = {0, 0};
    for (; at < end && max(have[0], have[1]) <= kCap - 64 * kU; at += 64 * kU) {
      int y[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) y[u] = at + 64 * u + lane < end ? p.live.y[at + 64 * u + lane] : -1;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t v = y[u] - v0;
        if (!__any(y[u] >= 0 && v >= 0 && v < 2 * kWave)) continue;
        const int t = at + 64 * u + lane;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bool in = y[u] >= 0 && v >= s * kWave && v < (s + 1) * kWave;
          const uint64_t mask = __ballot(in);
          if (in)
            list[(4 * s + wave) * kCap + have[s] + __popcll(mask & ((1ull << lane) - 1ull))] = {
                (uint32_t)t << 7 | (uint32_t)(v - s * kWave), lost_of(p.live.cy[t])};
          have[s] += __popcll(mask);
        }
      }
    }
    if (lane == 0) {
      count[wave] = have[0];
      count[4 + wave] = have[1];
      more[wave] = at < end;
    }
    __syncthreads();
    const int* const mine = count + 4 * half;
    const int c1 = mine[0], c2 = c1 + mine[1], c3 = c2 + mine[2], all = __builtin_amdgcn_readfirstlane(c3 + mine[3]);
    for (int k0 = 0; k0 < all; k0 += 16) {
      Found f[8];  // this lane's half of a product's slots
      uint32_t x[8][kF];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = min(k0 + 8 * h + u, all - 1);
        const int w = (i >= c1) + (i >= c2) + (i >= c3), first = w == 0 ? 0 : w == 1 ? c1 : w == 2 ? c2 : c3;
        f[u] = list[(4 * half + w) * kCap + i - first];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int g = 0; g < kF; ++g)  // columns past D are not stored
          x[u][g] = p.live.xr[(int64_t)(f[u].key >> 7) * p.Dx + min<int64_t>(d + 32 * g, p.D - 1)];
      uint32_t wb[kF][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t both = pack_bf16(f[2 * q].lost, f[2 * q + 1].lost);
        const int at0 = k0 + 8 * h + 2 * q;
        const int word0 = at0 < all ? (int)(f[2 * q].key & 127u) : -1, word1 = at0 + 1 < all ? (int)(f[2 * q + 1].key & 127u) : -1;
#pragma unroll
        for (int j = 0; j < kF; ++j)
          wb[j][q] = (word0 == 32 * j + l32 ? both & 0xFFFFu : 0u) | (word1 == 32 * j + l32 ? both & 0xFFFF0000u : 0u);
      }
#pragma unroll
      for (int g = 0; g < kF; ++g) {
        const uint4 wa = make_uint4(x[0][g] | x[1][g] << 16, x[2][g] | x[3][g] << 16, x[4][g] | x[5][g] << 16, x[6][g] | x[7][g] << 16);
#pragma unroll
        for (int j = 0; j < kF; ++j)
          acc[g][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(gemm::bf16x8, wa),
              __builtin_bit_cast(gemm::bf16x8, make_uint4(wb[j][0], wb[j][1], wb[j][2], wb[j][3])), acc[g][j], 0, 0, 0);
      }
    }
    const bool again = (more[0] | more[1] | more[2] | more[3]) != 0;
    __syncthreads();
    if (!again) return;
  }
}

// dw rows of the piece (32768 x 4096 out of 8192 tokens: 1.68 ms, 1.31 PFLOP/s).
template <int kF, bool kF32, bool kAdd>
__global__ __launch_bounds__(gemm::kThreads, kF == 4 ? 1 : 2) void k_ce_dw(CeParams p) {
  constexpr int kEdge = 64 * kF, kWave = 32 * kF;
  __shared__ __attribute__((aligned(16))) char lds[gemm::Shape<kF>::kLdsBytes];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n = *p.live.count;
  const float s = p.scale * *p.live.g;
  run_tile<kF, true, true, false>(
      p, p.v1 - p.v0, p.D, lds,
      [&](int64_t vt, int64_t d0, gemm::Panel& A, gemm::Panel& B) -> bool {
        if (d0 >= p.D || p.v0 + vt >= p.V) return false;  // a quarter outside
        A = {p.live.xr + d0, (uint32_t)p.Dx, (int)min<int64_t>(kEdge, p.D - d0), n};
        B = {p.c + vt, (uint32_t)p.Vp, kEdge, n};
        return true;
      },
      [&](int64_t vt, int64_t d0, f32x16 (&acc)[kF][kF]) {
        const int lane = lane_here(), l32 = lane & 31, h = lane >> 5;
        const int64_t dwv = d0 + kWave * (wave & 1), vw = p.v0 + vt + kWave * (wave >> 1);
        const int64_t rows = p.V - vw, cols = p.D - dwv;
        if (*p.live.uneven) add_targets<kF>(p, lds, (int)n, p.v0 + vt, d0, acc);
        if (!kF32 && !kAdd) {
          uint16_t* const out = static_cast<uint16_t*>(p.dw) + vw * p.dw_ld + dwv;
          store_block<kF>(
              lds + 2048 * kF * wave, acc,
              [&](int, float (&z)[kF][16]) {
#pragma unroll
                for (int i = 0; i < kF; ++i)
#pragma unroll
                  for (int v = 0; v < 16; ++v) z[i][v] *= s;
              },
              [&](int n, int c, uint4 q) {
                if (n < rows && 8 * c < cols) *reinterpret_cast<uint4*>(out + n * p.dw_ld + 8 * c) = q;
              });
          return;
        }
        // fp32, or added to what is there (rounded once): straight from the
        // accumulators, four neighbours a lane
#pragma unroll
        for (int j = 0; j < kF; ++j) {
          if (32 * j + l32 >= rows) continue;
#pragma unroll
          for (int i = 0; i < kF; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int d = row_of(i, 4 * q) + 4 * h;
              if (d >= cols) continue;
              const int64_t at = (vw + 32 * j + l32) * p.dw_ld + dwv + d;
              float r[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) r[k] = acc[i][j][4 * q + k] * s;
              if (kF32) {
                float4* const o = reinterpret_cast<float4*>(static_cast<float*>(p.dw) + at);
                const float4 old = kAdd ? *o : make_float4(0, 0, 0, 0);
                *o = kAdd ? make_float4(r[0] + old.x, r[1] + old.y, r[2] + old.z, r[3] + old.w)
                          : make_float4(r[0], r[1], r[2], r[3]);
              } else {
                uint2* const o = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dw) + at);
                const uint2 old = *o;
                *o = make_uint2(pack_bf16(r[0] + bf16_lo(old.x), r[1] + bf16_hi(old.x)),
                                pack_bf16(r[2] + bf16_lo(old.y), r[3] + bf16_hi(old.y)));
              }
            }
        }
      });
}

// ------------------------------------------------------------------- host --
// Entries of c at a time: 512 MB.  Any size that fills the card does (gradient of
// 8192 tokens, 65536 words of 4096: 2^26 / 2^28 / 2^30 entries 10.41 / 10.46 /
// 10.48 ms); small ones lose where tokens are many (16384 of 2048: 12.49 / 10.95 /
// 11.03 ms).
constexpr int64_t kPieceElements = (int64_t)1 << 28;
// Workgroups of the kernel for few tokens: two a CU, as many as fit (16 tokens,
// 65536 words of 4096: 256 / 512 / 768 workgroups 111 / 104 / 109 us).
constexpr int64_t kFewBlocks = 512;
constexpr int64_t kMaxCeTokens = (int64_t)1 << 23;
constexpr int64_t kMaxStride = (int64_t)1 << 21;      // elements: 256 rows of a panel stay below 2^31 bytes

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

struct CeLayout {
  CeParams p;
  int64_t piece;
  size_t bytes;
};

// Whether the forward takes the kernel for few tokens.  It reads w at what HBM
// gives up to 32 tokens (65536 words of 7168, 1 / 32 / 48 / 64 tokens: 160 / 180
// / 202 / 222 us; in tiles 206 / 201 / 204 / 208), and for some more where
// the tiles would leave CUs idle (32768 words of 2048: 27 / 30 / 36 / 38 us, in
// tiles 49 / 50 / 51 / 51).  Where few words leave idle CUs, more tokens go 64 at
// a time, as long as the workgroups fit one a CU (1000 tokens, 1000 words of 8192:
// 64 us, in tiles 91; 256, 4000 of 4096: 37 / 53; past that 512, 4000: 66 / 53;
// 100, 10000: 61 / 54).
bool few(int64_t T, int64_t V) {
  return T <= 48 || (T <= kFew && V <= 160 * kTile) || (T + kFew - 1) / kFew * ((V + 63) / 64) <= 256;
}

// Partial results that the forward leaves for each token: a workgroup's of the
// kernel for few tokens, else a tile's.
int64_t forward_parts(int64_t T, int64_t V) {
  return few(T, V) ? std::min<int64_t>((V + 63) / 64, kFewBlocks) : (V + kPart - 1) / kPart;
}

size_t forward_layout(void* ws, int64_t T, int64_t V, CeParams* p) {
  WsCarve c(ws);
  float2* const part = c.take<float2>((size_t)(forward_parts(T, V) * T));
  float* const at = c.take<float>((size_t)T);
  if (p) {
    p->part = part;
    p->at = at;
    p->status = c.status();
  }
  return c.off;
}

void backward_layout(void* ws, CeLayout& L) {
  CeParams& p = L.p;
  p.Tp = up(std::max<int64_t>(p.T, 1), kTile);
  p.Dx = up(p.D, 64) + 64;
  // pieces of equal length, whole tiles of the vocabulary
  const int64_t tiles = (p.V + kTile - 1) / kTile;
  const int64_t most = std::max<int64_t>(1, kPieceElements / (p.Tp * kTile));
  const int64_t pieces = (tiles + most - 1) / most;
  L.piece = (tiles + pieces - 1) / pieces * kTile;
  p.Vp = L.piece + 64;
  // dx: one workgroup a CU (gradient of 1023 tokens, 50001 words of 1000 for 128 /
  // 256 / 512: 404 / 377 / 436 us; 300, 128000 of 4096: 1745 / 1444 / 1466), each
  // with at least 256 words
  const int64_t dx_tiles = p.Tp / kTile * ((p.D + kTile - 1) / kTile);
  p.slices = (int)std::max<int64_t>(1, std::min<int64_t>(256 / dx_tiles, L.piece / 256));
  WsCarve c(ws);
  p.live.count = c.take<int32_t>(1);
  p.live.g = c.take<float>(1);
  p.live.row = c.take<int32_t>((size_t)p.T);
  p.live.pos = c.take<int32_t>((size_t)p.T);
  p.live.x = c.take<uint16_t>((size_t)(p.Tp * p.Dx));
  p.live.xr = c.take<uint16_t>((size_t)(p.Tp * p.Dx));
  p.live.m = c.take<float>((size_t)p.Tp);
  p.live.l2 = c.take<float>((size_t)p.Tp);
  p.live.y = c.take<int32_t>((size_t)p.Tp);
  p.live.cy = c.take<float>((size_t)p.T);
  p.live.uneven = c.take<int32_t>(1);
  p.c = c.take<uint16_t>((size_t)(p.Tp * p.Vp));
  p.slab = c.take<float>((size_t)(p.slices * p.Tp * p.D));
  p.status = c.status();
  L.bytes = c.off;
}

// The last: a launch of the forward's tiles stays below 2^32 threads.
bool ce_shape_ok(int64_t T, int64_t D, int64_t V) {
  return T >= 0 && T <= kMaxCeTokens && D >= 8 && D <= 65536 && D % 8 == 0 && V >= 1 && V <= ((int64_t)1 << 24) &&
         up(T, kTile) / kTile * (up(V, kTile) / kTile) <= ((int64_t)1 << 23);
}

// Launches a product's tiles: whole rounds of one tile of 256 a CU, and what is
// left over as quarters where those fit the CUs at once, two each.  2048 tokens,
// forward, 256 tiles and 16 / 80 / 112 / 144 / 208 more: of 4096 160 / 166 / 171 /
// 218 / 225 us in quarters, 184 / 187 / 190 / 193 / 203 as whole tiles; of 1024 55
// / 57 / 57 / 72 / 74 us against 62 / 63 / 63 / 66 / 68.
template <class K>
int launch_tiles(CeParams p, int64_t tiles, K whole, K quarters, hipStream_t s) {
  const int64_t cus = device_cu_count(), left = tiles % cus;
  const int64_t split = left <= cus / 2 ? tiles - left : tiles;
  p.tile0 = 0;
  p.tile1 = (int)split;
  if (split) {
    hipLaunchKernelGGL(whole, dim3(grid_of(split)), dim3(gemm::kThreads), 0, s, p);
    if (int rc = last_launch()) return rc;
  }
  p.tile0 = (int)split;
  p.tile1 = (int)tiles;
  if (split == tiles) return NVQ_OK;
  hipLaunchKernelGGL(quarters, dim3(grid_of(4 * (tiles - split))), dim3(gemm::kThreads), 0, s, p);
  return last_launch();
}

int check(const nvq_linear_ce_args* a, CeParams& p) {
  if (!a || a->struct_size < sizeof(nvq_linear_ce_args)) return NVQ_EINVAL;
  if (!ce_shape_ok(a->T, a->D, a->V)) return NVQ_ESHAPE;
  if (!a->w || (a->T && (!a->x || !a->targets))) return NVQ_EINVAL;
  if (!std::isfinite(a->scale)) return NVQ_EINVAL;
  p = CeParams{};
  p.T = a->T; p.D = a->D; p.V = a->V;
  p.x_ld = a->x_ld ? a->x_ld : a->D;
  p.w_ld = a->w_ld ? a->w_ld : a->D;
  if (p.x_ld < a->D || p.w_ld < a->D || p.x_ld > kMaxStride || p.w_ld > kMaxStride) return NVQ_ESHAPE;
  if (!aligned16(a->x) || !aligned16(a->w) || p.x_ld % 8 || p.w_ld % 8 || ((uintptr_t)a->targets & 3u) ||
      ((uintptr_t)a->loss & 3u) || ((uintptr_t)a->lse & 3u) || ((uintptr_t)a->dloss & 3u))
    return NVQ_EALIGN;
  p.x = a->x; p.w = a->w; p.targets = a->targets; p.scale = a->scale;
  p.loss = a->loss; p.lse = a->lse; p.dloss = a->dloss;
  return NVQ_OK;
}

}  // namespace
}  // namespace nvq

using namespace nvq;

extern "C" size_t nvq_linear_cross_entropy_workspace_bytes(int64_t T, int64_t D, int64_t V) {
  return ce_shape_ok(T, D, V) ? forward_layout(nullptr, T, V, nullptr) : kAlign;
}

extern "C" size_t nvq_linear_cross_entropy_backward_workspace_bytes(int64_t T, int64_t D, int64_t V) {
  if (!ce_shape_ok(T, D, V)) return kAlign;
  CeLayout L{};
  L.p.T = T; L.p.D = D; L.p.V = V;
  backward_layout(nullptr, L);
  return L.bytes;
}

extern "C" int nvq_linear_cross_entropy(const nvq_linear_ce_args* a, void* stream) {
  CeParams p;
  if (int rc = check(a, p)) return rc;
  if (!a->loss && !a->lse && a->T) return NVQ_EINVAL;
  if (!a->ws || a->ws_bytes < forward_layout(a->ws, p.T, p.V, &p)) return NVQ_EWORKSPACE;
  if (!aligned256(a->ws)) return NVQ_EALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (p.T == 0) return clear_status(p.status, s);
  const int64_t parts = forward_parts(p.T, p.V);
  if (few(p.T, p.V)) {
    auto k = p.T <= 16 ? k_ce_few<1> : p.T <= 32 ? k_ce_few<2> : k_ce_few<4>;
    hipLaunchKernelGGL(k, dim3((unsigned)parts, (unsigned)((p.T + kFew - 1) / kFew)), dim3(256), 0, s, p);
    if (int rc = last_launch()) return rc;
  } else if (int rc = launch_tiles(p, (p.V + kTile - 1) / kTile * ((p.T + kTile - 1) / kTile),
                                 p.T <= kTile ? k_ce_forward<4, true> : k_ce_forward<4, false>, k_ce_forward<2, false>, s)) {
    return rc;
  }
  hipLaunchKernelGGL(k_ce_join, dim3((unsigned)((p.T + 7) / 8)), dim3(1024), 0, s, p, (int)parts);
  return last_launch();
}

extern "C" int nvq_linear_cross_entropy_backward(const nvq_linear_ce_args* a, void* stream) {
  CeLayout L{};
  CeParams& p = L.p;
  if (int rc = check(a, p)) return rc;
  if (!a->dx && !a->dw) return NVQ_EINVAL;
  if (a->T && !a->lse) return NVQ_EINVAL;
  if (a->dw_dtype != NVQ_F32 && a->dw_dtype != NVQ_BF16) return NVQ_EINVAL;
  p.dx_ld = a->dx_ld ? a->dx_ld : p.D;
  p.dw_ld = a->dw_ld ? a->dw_ld : p.D;
  if (p.dx_ld < p.D || p.dw_ld < p.D) return NVQ_ESHAPE;
  const bool f32 = a->dw_dtype == NVQ_F32;
  if (!aligned16(a->dx) || !aligned16(a->dw) || p.dx_ld % 8 || p.dw_ld % (f32 ? 4 : 8)) return NVQ_EALIGN;
  backward_layout(a->ws, L);
  if (!a->ws || a->ws_bytes < L.bytes) return NVQ_EWORKSPACE;
  if (!aligned256(a->ws)) return NVQ_EALIGN;
  p.dx = a->dx; p.dw = a->dw;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(k_ce_live, dim3(1), dim3(1024), 0, s, p);
  if (int rc = last_launch()) return rc;
  const int64_t nt = p.Tp / kTile, nd = (p.D + kTile - 1) / kTile;
  if (p.T) {
    hipLaunchKernelGGL(k_ce_gather, dim3((unsigned)p.Tp), dim3(256), 0, s, p);
    if (int rc = last_launch()) return rc;
  }
  auto dw4 = f32 ? (a->accumulate ? k_ce_dw<4, true, true> : k_ce_dw<4, true, false>)
                 : (a->accumulate ? k_ce_dw<4, false, true> : k_ce_dw<4, false, false>);
  auto dw2 = f32 ? (a->accumulate ? k_ce_dw<2, true, true> : k_ce_dw<2, true, false>)
                 : (a->accumulate ? k_ce_dw<2, false, true> : k_ce_dw<2, false, false>);
  for (p.v0 = 0; p.v0 < p.V; p.v0 = p.v1) {
    p.v1 = std::min(p.v0 + L.piece, p.V);
    p.first = p.v0 == 0;
    const int64_t nv = (p.v1 - p.v0 + kTile - 1) / kTile;
    if (p.T)
      if (int rc = launch_tiles(p, nv * nt, nt == 1 ? k_ce_coef<4, true> : k_ce_coef<4, false>,
                                nt == 1 ? k_ce_coef<2, true> : k_ce_coef<2, false>, s))
        return rc;
    if (p.T && p.dx) {
      p.tile0 = 0;
      p.tile1 = (int)(nt * nd);
      hipLaunchKernelGGL(k_ce_dx, dim3(grid_of(nt * nd * p.slices)), dim3(gemm::kThreads), 0, s, p);
      if (int rc = last_launch()) return rc;
    }
    if (p.dw)
      if (int rc = launch_tiles(p, nv * nd, dw4, dw2, s)) return rc;
  }
  if (!p.T || !p.dx) return NVQ_OK;
  const bool split = p.slices >= 8;
  hipLaunchKernelGGL(split ? k_ce_dx_join<true> : k_ce_dx_join<false>,
                     dim3((unsigned)p.T, (unsigned)((p.D + (split ? 255 : 1023)) / (split ? 256 : 1024))), dim3(256), 0, s, p);
  return last_launch();
}
