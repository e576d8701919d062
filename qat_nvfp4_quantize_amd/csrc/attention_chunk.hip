// Attention over the paged NVFP4 cache for sequences of many query rows per
// key/value head (prompt chunks): bound by the matrix cores and the softmax's
// exponentials, so a tile of keys is dequantized once for 128 rows.
//
// A workgroup takes 128 (token, head-of-the-group) rows of one sequence and
// key/value head, a wave 32 of them, over 64 keys at a time.  The keys' codes
// come into registers one tile ahead, are dequantized exactly to fp16 and
// written row-major to LDS (K and V alike, double-buffered, one barrier a
// tile).  Products run transposed (32x32x16 fp16): S^T = K Q^T leaves a lane
// one query and 16 keys of each 32, which is already the B operand of O^T =
// V^T P^T; the A operand comes out of the row-major V tile through LDS
// transpose reads.  The softmax reference moves only when a score exceeds it
// by 15 (powers of two), as in the few-rows kernel.
//
// Row tiles with many keys are split over workgroups where there are few of
// them (planned on the device from cu_q and kv_len), and joined afterwards.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "nvq.h"
#include "nvq_attn.h"
#include "nvq_dequant.h"
#include "nvq_device.h"
#include "nvq_internal.h"
#include "nvq_scan.h"

namespace nvq {
namespace {

typedef float floatx16_t __attribute__((ext_vector_type(16)));
typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef short v8i16_t __attribute__((ext_vector_type(8)));
#define NVQ_LDS __attribute__((address_space(3)))

constexpr int kTileRows = 128, kTileKeys = 64;
constexpr float kRefRoom = 15, kRefStart = 9;  // as in the few-rows kernel

// Keys of row tile qt of sequence s, in 64-key tiles from `base`.
struct TileRange {
  int64_t base, hi;
  int units;
};
__device__ __forceinline__ TileRange tile_range(const AttnParams& p, const Seq& s, int qt) {
  const int i0 = (int)((int64_t)qt * kTileRows / p.g);
  const int i1 = min(s.n - 1, (int)(((int64_t)(qt + 1) * kTileRows - 1) / p.g));
  TileRange r;
  int64_t lo, x;
  visible(p, s, s.pos0 + i0, lo, x);
  visible(p, s, s.pos0 + i1, x, r.hi);
  r.base = lo & ~(int64_t)(kTileKeys - 1);
  r.units = r.hi > r.base ? (int)((r.hi - r.base + kTileKeys - 1) / kTileKeys) : 1;
  return r;
}

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* s_wave) {
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) v += __shfl_xor(v, x, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6] = v;
  __syncthreads();
  int64_t sum = 0;
  for (int w = 0; w < (int)blockDim.x >> 6; ++w) sum += s_wave[w];
  return sum;
}

// One workgroup plans the call: the row tiles of the sequences (the last rows,
// which see the most keys, first), their pieces, and the list of split tiles.
__global__ __launch_bounds__(1024) void k_attn_chunk_plan(AttnParams p, ChunkPlan plan) {
  __shared__ int64_t s_sum[16];
  __shared__ int s_scan[16];
  __shared__ int s_last;
  const int t = threadIdx.x;
  auto last = [&](int incl) {  // the workgroup's total of an inclusive scan
    __syncthreads();
    if (t == 1023) s_last = incl;
    __syncthreads();
    return s_last;
  };
  int tiles = 0;
  for (int b0 = 0; b0 < p.B; b0 += 1024) {
    int n = 0;
    if (b0 + t < p.B) {
      const Seq s = load_seq(p, b0 + t);
      const int64_t rows = (int64_t)s.n * p.g;
      n = rows > plan.min_rows ? (int)((rows + kTileRows - 1) / kTileRows) : 0;
    }
    const int incl = block_inclusive_scan(n, s_scan);
    if (b0 + t < p.B) plan.tile_end[b0 + t] = tiles + incl;
    tiles += last(incl);
  }
  tiles = min<int64_t>(tiles, plan.max_tiles);  // overlapping row ranges could name more
  __threadfence_block();
  __syncthreads();
  auto tile_at = [&](int i, int& b, int& qt) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (plan.tile_end[mid] > i)
        hi = mid;
      else
        lo = mid + 1;
    }
    b = lo;
    qt = plan.tile_end[lo] - 1 - i;
    return tile_range(p, load_seq(p, lo), qt).units;
  };
  int64_t total = 0;
  for (int i = t; i < tiles; i += 1024) {
    int b, qt;
    total += tile_at(i, b, qt);
  }
  total = block_sum(total, s_sum);
  const int64_t per = max<int64_t>((total * p.c.H + plan.target - 1) / plan.target, plan.min_units);
  int items = 0, slots = 0, splits = 0;
  for (int i0 = 0; i0 < tiles; i0 += 1024) {
    int b = 0, qt = 0, n = 0;
    if (i0 + t < tiles) n = (int)((tile_at(i0 + t, b, qt) + per - 1) / per);
    const int split = n > 1;
    const int incl = block_inclusive_scan(n, s_scan);
    const int all = last(incl);
    const int incl_slot = block_inclusive_scan(split ? n : 0, s_scan);
    const int all_slot = last(incl_slot);
    const int incl_split = block_inclusive_scan(split, s_scan);
    const int all_split = last(incl_split);
    for (int k = 0; k < n; ++k)
      plan.item[items + incl - n + k] = make_int4(b, qt, k << 16 | n, slots + incl_slot - n + k);
    if (split) plan.split[splits + incl_split - 1] = make_int4(b, qt, n, slots + incl_slot - n);
    items += all, slots += all_slot, splits += all_split;
  }
  if (t == 0) plan.count[0] = items, plan.count[1] = splits;
}

// Two transpose reads -> the 8 keys of one element of an A operand: in each
// group of 16 lanes, lane i receives element i % 4 of the 8-byte reads of
// lanes i / 4 + 4 m, m = 0..3.
__device__ __forceinline__ half8_t tr_pair(const NVQ_LDS char* at, int second) {
  const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((NVQ_LDS v4i16_t*)at);
  const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((NVQ_LDS v4i16_t*)(at + second));
  const v8i16_t v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(half8_t, v);
}

// Codes and scales of a quarter of one key's elements, K and V.
template <int D>
struct TileRegs {
  uint32_t k[D / 32], v[D / 32], ks[D / 128], vs[D / 64];
};
template <>
struct TileRegs<64> {
  uint32_t k[2], v[2], ks, vs;
};

// A wave loads 16 keys of a tile, which lie in one page: its base is uniform,
// and a lane's offsets in it (key16 of the 16 keys, quarter `part` of the
// elements) never change.  id < 0 (no such page) reads page 0, masked later.
template <int D>
__device__ __forceinline__ void load_tile(const AttnParams& p, TileRegs<D>& r, int id, int kvh, int off,
                                          uint32_t key16, uint32_t part) {
  const int64_t tile = ((int64_t)max(id, 0) * p.c.H + kvh) << p.c.log_ps;
  const uint8_t* kc = p.c.k_codes + (tile + off) * (D / 2);
  const uint8_t* vc = p.c.v_codes + (tile + off) * (D / 2);
  const uint8_t* ks = p.c.k_scales + (tile + off) * (D / 16);
  const uint8_t* vs = p.c.v_scales + tile * (D / 16) + off;
  const uint32_t at = key16 * (D / 2), sat = key16 * (D / 16);
  if constexpr (D == 64) {
    const uint2 x = *reinterpret_cast<const uint2*>(kc + (at + 8 * part));
    const uint2 y = *reinterpret_cast<const uint2*>(vc + (at + 8 * part));
    r.k[0] = x.x, r.k[1] = x.y, r.v[0] = y.x, r.v[1] = y.y;
    r.ks = ks[sat + part];
    r.vs = vs[key16 + (part << p.c.log_ps)];
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(kc + (at + 16 * part) + 64 * i);
      const uint4 y = *reinterpret_cast<const uint4*>(vc + (at + 16 * part) + 64 * i);
      r.k[4 * i] = x.x, r.k[4 * i + 1] = x.y, r.k[4 * i + 2] = x.z, r.k[4 * i + 3] = x.w;
      r.v[4 * i] = y.x, r.v[4 * i + 1] = y.y, r.v[4 * i + 2] = y.z, r.v[4 * i + 3] = y.w;
      r.ks[i] = *reinterpret_cast<const uint16_t*>(ks + (sat + 2 * part) + 8 * i);
      r.vs[2 * i] = vs[key16 + ((8 * i + 2 * part) << p.c.log_ps)];
      r.vs[2 * i + 1] = vs[key16 + ((8 * i + 2 * part + 1) << p.c.log_ps)];
    }
  }
}

// Byte of an E4M3 scale -> fp16 pair s_b * 2^-8, finite for any byte.
__device__ __forceinline__ uint32_t scale_of(uint32_t byte) { return (byte & 0x7Fu) * 0x00800080u; }

// Dequantizes and writes to the LDS tiles.
template <int D>
__device__ __forceinline__ void store_tile(const TileRegs<D>& r, uint8_t* k, uint8_t* v, int part) {
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    const int at = D == 64 ? 32 * part + 16 * j : 256 * (j >> 2) + 64 * part + 16 * (j & 3);
    uint32_t ks, vs;
    if constexpr (D == 64)
      ks = scale_of(r.ks), vs = scale_of(r.vs);
    else
      ks = scale_of((j >> 1) & 1 ? r.ks[j >> 2] >> 8 : r.ks[j >> 2]), vs = scale_of(r.vs[j >> 1]);
    *reinterpret_cast<half8_t*>(k + at) = dequant8(r.k[j], ks);
    *reinterpret_cast<half8_t*>(v + at) = dequant8(r.v[j], vs);
  }
}

// A tile in LDS: key k at (k % 4) kPlane + (k / 4) kRow.  Rows are 16 bytes past
// a multiple of 256 (128 for D = 64) and planes 64, so that each access of 256
// bytes a clock meets every bank once: the 16 keys of a 16-byte read, the 4
// keys x 64 bytes of a transpose read, and the loader's writes (whose 16 lanes
// take keys 4 apart).  A plain pitch of 2 D + 32 cost a quarter of the time in
// bank conflicts.
template <int D>
struct ChunkLds {
  static constexpr int kRow = 2 * D + 16, kPlane = kTileKeys / 4 * kRow + 64;
  static constexpr int kTile = 3 * kPlane + kTileKeys / 4 * kRow;
  alignas(16) uint8_t k[2][kTile];
  alignas(16) uint8_t v[2][kTile];
  alignas(16) uint32_t dead[2][4];  // 16 keys without a page
  static __device__ __forceinline__ int at(int key) { return (key & 3) * kPlane + (key >> 2) * kRow; }
};

// Largest of three (v_max3_f32; fmaxf would first quiet each operand).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(m) : "v"(a), "v"(b), "v"(c));
  return m;
}

template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_attn_chunk(AttnParams p, ChunkPlan plan) {
  using Lds = ChunkLds<D>;
  constexpr int kSteps = D / 16, kOut = D / 32;
  __shared__ Lds lds;
  if (plan.check && blockIdx.x == 0) {
    check_batch(p, reinterpret_cast<CheckLds&>(lds));
    return;
  }
  const int block = blockIdx.x - plan.check, kvh = block % p.c.H, item = block / p.c.H;
  if (item >= plan.count[0]) return;
  const int4 it = plan.item[item];
  const int b = __builtin_amdgcn_readfirstlane(it.x), qt = __builtin_amdgcn_readfirstlane(it.y);
  const int index = __builtin_amdgcn_readfirstlane(it.z) >> 16, count = __builtin_amdgcn_readfirstlane(it.z) & 0xFFFF;
  const Seq s = load_seq(p, b);
  const TileRange range = tile_range(p, s, qt);
  const int u_begin = (int)((int64_t)index * range.units / count);
  const int u_end = (int)((int64_t)(index + 1) * range.units / count);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, h = lane >> 5;
  const int32_t* table = p.table + b * p.table_ld;

  // this lane's query row
  const int64_t rows = (int64_t)s.n * p.g, r = (int64_t)qt * kTileRows + 32 * wave + l32;
  const bool live = r >= 0 && r < rows;
  const int qi = live ? (int)(r / p.g) : 0, qh = kvh * p.g + (live ? (int)(r % p.g) : 0);
  half8_t qf[kSteps];
  float cq;
  {
    const uint16_t* at = p.q + (s.row0 + qi) * p.q_ld_t + qh * p.q_ld_h + 8 * h;
    uint32_t w[kSteps][4], top = 0;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const uint4 x = *reinterpret_cast<const uint4*>(at + 16 * u);
      w[u][0] = x.x, w[u][1] = x.y, w[u][2] = x.z, w[u][3] = x.w;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max(w[u][j] << 16 & 0x7FFF0000u, w[u][j] & 0x7FFF0000u));
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    // as in the few-rows kernel; the sign of the factor goes into Q, so that
    // the largest product is the largest score, and a factor of 0 too
    const int ex = (int)(top >> 23);
    const int shift = (top == 0u || ex == 255) ? 0 : 14 + 127 - max(ex, 1);
    const float c0 = __builtin_ldexpf(p.scale_log2 * *p.c.k_st, -shift);
    const float sign = c0 < 0.0f ? -1.0f : c0 > 0.0f ? 1.0f : 0.0f;
    cq = c0 == 0.0f ? 1.0f : fabsf(c0);
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        qf[u][2 * j] = (_Float16)(__builtin_ldexpf(bf16_lo(w[u][j]), shift) * sign);
        qf[u][2 * j + 1] = (_Float16)(__builtin_ldexpf(bf16_hi(w[u][j]), shift) * sign);
      }
  }
  int64_t lo64, hi64;
  visible(p, s, s.pos0 + qi, lo64, hi64);
  const int see_lo = (int)min<int64_t>(lo64, INT32_MAX), see_hi = live ? (int)max<int64_t>(hi64, 0) : 0;
  // every row of the wave sees all of [all_lo, all_hi)
  const int64_t r0 = (int64_t)qt * kTileRows + 32 * wave;
  int64_t all_lo, all_hi, x64;
  visible(p, s, s.pos0 + min(r0, rows - 1) / p.g, x64, all_hi);
  visible(p, s, s.pos0 + min(r0 + 31, rows - 1) / p.g, all_lo, x64);

  floatx16_t o[kOut];
#pragma unroll
  for (int i = 0; i < kOut; ++i) o[i] = (floatx16_t)(0.0f);
  float ref = -INFINITY, ref_safe = 0.0f, l = 0.0f;

  // Loader: a wave takes 16 keys of the tile, a thread a quarter of one of
  // them, 16 lanes keys 4 apart.  Page ids of the wave's next 64 tiles with one
  // load (-1: no key, or an id outside the cache).
  const int part = threadIdx.x & 3, key16 = 4 * ((lane >> 2) & 3) + (lane >> 4);
  const int lkey_at = Lds::at(16 * wave + key16);
  const int64_t base = range.base + 16 * wave;
  int ids = -1, ids_at = u_begin;
  auto fetch_ids = [&](int u0) {
    const int64_t key = base + (int64_t)(u0 + lane) * kTileKeys;
    const int id = (u0 + lane < u_end && key < range.hi) ? table[key >> p.c.log_ps] : -1;
    ids = id < p.c.num_pages ? id : -1;
    ids_at = u0;
  };
  TileRegs<D> regs;
  int id;
  auto fetch = [&](int u) {  // past the last tile: page 0, never looked at
    if (u - ids_at >= 64) fetch_ids(u);
    id = __builtin_amdgcn_readlane(ids, u - ids_at);
    load_tile<D>(p, regs, id, kvh, (int)(base + (int64_t)u * kTileKeys) & (p.c.ps - 1), key16, part);
  };
  auto put = [&](int buf) {
    store_tile<D>(regs, lds.k[buf] + lkey_at, lds.v[buf] + lkey_at, part);
    if (lane == 0) lds.dead[buf][wave] = id < 0;
  };
  fetch_ids(u_begin);
  fetch(u_begin);
  put(0);
  __syncthreads();

  // lane's source address of a transpose read: key 4 h + s / 4, elements
  // 16 (lane / 16 % 2) + 4 (s % 4), s = lane % 16
  const int tr_off = Lds::at(4 * h + ((lane & 15) >> 2)) + 2 * (16 * ((lane >> 4) & 1) + 4 * (lane & 3));
#pragma unroll 1
  for (int u = u_begin; u < u_end; ++u) {
    const int buf = (u - u_begin) & 1;
    const int64_t kb = range.base + (int64_t)u * kTileKeys;
    fetch(u + 1);
    floatx16_t sc[2];
    const uint8_t* k_at = lds.k[buf] + Lds::at(l32) + 16 * h;
    sc[0] = sc[1] = (floatx16_t)(0.0f);
#pragma unroll
    for (int w = 0; w < kSteps; ++w)
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)  // two chains of products in turn
        sc[kt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            *reinterpret_cast<const half8_t*>(k_at + 8 * kt * Lds::kRow + 32 * w), qf[w], sc[kt], 0, 0, 0);
    const uint4 dead = *reinterpret_cast<const uint4*>(lds.dead[buf]);
    if (kb < all_lo || kb + kTileKeys > all_hi || (dead.x | dead.y | dead.z | dead.w)) {
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int k = 32 * kt + 8 * (v >> 2) + 4 * h + (v & 3), key = (int)kb + k;
          const uint32_t none = 2 * kt + (v >> 3) == 0 ? dead.x : 2 * kt + (v >> 3) == 1 ? dead.y
                                : 2 * kt + (v >> 3) == 2 ? dead.z : dead.w;
          sc[kt][v] = (key >= see_lo && key < see_hi && !none) ? sc[kt][v] : -INFINITY;
        }
    }
    float top = max3(sc[0][0], sc[1][0], sc[1][1]), top2 = max3(sc[0][1], sc[0][2], sc[1][2]);
#pragma unroll
    for (int v = 3; v < 15; v += 2) {
      top = max3(top, sc[0][v], sc[1][v]);
      top2 = max3(top2, sc[0][v + 1], sc[1][v + 1]);
    }
    top = max3(top, sc[0][15], sc[1][15]);
    top = fmaxf(top, top2);
    top *= cq;
    if (__ballot(top > ref + kRefRoom)) {
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float moved = top > ref + kRefRoom ? top - kRefStart : ref;
      const float keep = moved == ref ? 1.0f : __builtin_amdgcn_exp2f(ref - moved);
      ref = moved;
      ref_safe = moved == -INFINITY ? 0.0f : moved;
      l *= keep;
#pragma unroll
      for (int i = 0; i < kOut; ++i) o[i] *= keep;
    }
    half8_t pf[4];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[kt][v], cq, -ref_safe));
        l += w;
        pf[2 * kt + (v >> 3)][v & 7] = (_Float16)w;
      }
    const NVQ_LDS char* vt = (const NVQ_LDS char*)lds.v[buf] + tr_off;
#pragma unroll
    for (int i = 0; i < kOut; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(tr_pair(vt + 4 * j * Lds::kRow + 64 * i, 2 * Lds::kRow), pf[j], o[i],
                                                      0, 0, 0);
    put(buf ^ 1);
    __syncthreads();
  }

  l += __shfl_xor(l, 32, 64);
  if (count == 1) {
    if (!live) return;
    const float inv = l == 0.0f ? 0.0f : *p.c.v_st / l;
    uint16_t* out = p.out + (s.row0 + qi) * p.out_ld_t + qh * p.out_ld_h;
#pragma unroll
    for (int i = 0; i < kOut; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        *reinterpret_cast<uint2*>(out + 32 * i + 8 * v + 4 * h) =
            make_uint2(f32_to_bf16_any(o[i][4 * v] * inv) | (f32_to_bf16_any(o[i][4 * v + 1] * inv) << 16),
                       f32_to_bf16_any(o[i][4 * v + 2] * inv) | (f32_to_bf16_any(o[i][4 * v + 3] * inv) << 16));
    if (p.lse && h == 0)
      p.lse[(int64_t)(s.row0 + qi) * p.Hq + qh] = l == 0.0f ? -INFINITY : (ref + __builtin_log2f(l)) * kLn2;
  } else {
    const int64_t slot = ((int64_t)__builtin_amdgcn_readfirstlane(it.w) * p.c.H + kvh) * kTileRows + 32 * wave + l32;
    float* out = plan.part_o + slot * D;
#pragma unroll
    for (int i = 0; i < kOut; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        *reinterpret_cast<float4*>(out + 32 * i + 8 * v + 4 * h) =
            make_float4(o[i][4 * v], o[i][4 * v + 1], o[i][4 * v + 2], o[i][4 * v + 3]);
    if (h == 0) plan.part_ml[slot] = make_float2(ref, l);
  }
}

// Joins the pieces of the split row tiles: a wave per row, a lane D / 64
// elements; the workgroups walk the (tile, head, 4 rows) list.
template <int D>
__global__ __launch_bounds__(256) void k_attn_chunk_join(AttnParams p, ChunkPlan plan) {
  constexpr int kE = D / 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t todo = (int64_t)plan.count[1] * p.c.H * (kTileRows / 4);
  for (int64_t w = blockIdx.x; w < todo; w += gridDim.x) {
    const int rr = (int)(w % (kTileRows / 4)) * 4 + wave;
    const int64_t th = w / (kTileRows / 4);
    const int kvh = (int)(th % p.c.H);
    const int4 it = plan.split[th / p.c.H];
    const Seq s = load_seq(p, it.x);
    const int64_t r = (int64_t)it.y * kTileRows + rr;
    if (r >= (int64_t)s.n * p.g) continue;
    auto slot = [&](int i) { return ((int64_t)(it.w + i) * p.c.H + kvh) * kTileRows + rr; };
    float m = -INFINITY;
    for (int i = lane; i < it.z; i += 64) m = fmaxf(m, plan.part_ml[slot(i)].x);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x, 64));
    const float ref = m == -INFINITY ? 0.0f : m;
    float o[kE], l = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = 0.0f;
#pragma unroll 4
    for (int i = 0; i < it.z; ++i) {
      const float2 ml = plan.part_ml[slot(i)];
      const float f = __builtin_amdgcn_exp2f(ml.x - ref);
      l += ml.y * f;
#pragma unroll
      for (int e = 0; e < kE; ++e) o[e] += plan.part_o[slot(i) * D + kE * lane + e] * f;
    }
    const int qi = (int)(r / p.g), qh = kvh * p.g + (int)(r % p.g);
    const float inv = l == 0.0f ? 0.0f : *p.c.v_st / l;
    uint16_t* out = p.out + (s.row0 + qi) * p.out_ld_t + qh * p.out_ld_h + kE * lane;
#pragma unroll
    for (int e = 0; e < kE; ++e) out[e] = (uint16_t)f32_to_bf16_any(o[e] * inv);
    if (p.lse && lane == 0)
      p.lse[(int64_t)(s.row0 + qi) * p.Hq + qh] = l == 0.0f ? -INFINITY : (m + __builtin_log2f(l)) * kLn2;
  }
}

template <int D>
int launch_chunk(const AttnParams& p, const ChunkPlan& plan, hipStream_t s) {
  hipLaunchKernelGGL(k_attn_chunk_plan, dim3(1), dim3(1024), 0, s, p, plan);
  if (int rc = last_launch()) return rc;
  hipLaunchKernelGGL((k_attn_chunk<D>), dim3((unsigned)(plan.max_items * p.c.H + plan.check)), dim3(256), 0, s, p,
                     plan);
  if (int rc = last_launch()) return rc;
  if (!plan.may_split) return NVQ_OK;
  hipLaunchKernelGGL((k_attn_chunk_join<D>), dim3(2 * device_cu_count()), dim3(256), 0, s, p, plan);
  return last_launch();
}

}  // namespace

void attn_chunk_plan(const AttnParams& p, int min_rows, bool check, WsCarve& ws, ChunkPlan& plan) {
  plan.min_rows = min_rows;
  plan.min_units = kChunkMinUnits;
  plan.target = kChunkTarget;
  plan.check = check;
  // rows of a sequence are cut to the call's, so its tiles are at most this
  plan.max_tiles = (int64_t)p.total_q * p.g / kTileRows + p.B;
  const int64_t units = (p.num_keys + 2 * kTileKeys - 2) / kTileKeys;
  plan.may_split = units > plan.min_units;
  const int64_t by_target = (plan.target + p.c.H - 1) / p.c.H;
  plan.max_items = plan.max_tiles + (plan.may_split ? by_target : 0);
  plan.count = ws.take<int32_t>(2);
  plan.tile_end = ws.take<int32_t>((size_t)p.B);
  plan.item = ws.take<int4>((size_t)plan.max_items);
  // ceil(units / per) > 1 pieces are at most 2 units / per
  const int64_t slots = plan.may_split ? std::min(2 * by_target, plan.max_items) : 0;
  plan.split = ws.take<int4>((size_t)slots);
  plan.part_ml = ws.take<float2>((size_t)(slots * p.c.H * kTileRows));
  plan.part_o = ws.take<float>((size_t)(slots * p.c.H * kTileRows * p.c.D));
}

int attn_chunk_launch(const AttnParams& p, const ChunkPlan& plan, hipStream_t s) {
  switch (p.c.D) {
    case 64: return launch_chunk<64>(p, plan, s);
    case 128: return launch_chunk<128>(p, plan, s);
    default: return launch_chunk<256>(p, plan, s);
  }
}

}  // namespace nvq
