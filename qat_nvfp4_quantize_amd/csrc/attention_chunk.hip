// Attention over the paged NVFP4 cache for sequences of many query rows per
// key/value head (prompt chunks): compute-bound, so a tile of keys is
// dequantized once for 128 or 256 rows.
//
// A workgroup takes 128 (token, head-of-the-group) rows of one sequence and
// key/value head (256 at head dimension 128 and many keys), a wave 32 of them,
// over 64 keys at a time.  The keys' codes
// come into registers one tile ahead, are dequantized exactly to fp16 and
// written row-major to LDS (K and V alike, double-buffered, one barrier a
// tile).  Products run transposed (32x32x16 fp16): S^T = K Q^T leaves a lane
// one query and 16 keys of each 32, which is already the B operand of O^T =
// V^T P^T; the A operand comes out of the row-major V tile through LDS
// transpose reads.  The softmax reference moves only when a score exceeds it
// by 15 (powers of two), and the weights are rounded to fp16, as in the few-rows
// kernel.
//
// Measured: two chunks of 4096 tokens behind 4096 and 2562 keys, 32 heads on 8
// of 128, 720 us, 1.0 PFLOP/s.  The same products and operand reads in a loop
// of their own, with six vector operations a product, reach 1.4 (the products
// alone 1.5): with such operands the card lowers its clock, so what counts is
// the number of operations, and orders of them that overlap better (the next
// tile's scores under this one's softmax, operands read three steps ahead, 64
// rows a wave, a barrier every second tile) measured 0 to 10 % slower.
//
// Where there are few row tiles, their key tiles are dealt to the workgroups
// that the chip holds in equal runs (planned on the device from cu_q and
// kv_len), and the parts of tiles that a run's end divides are joined.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "nvq.h"
#include "nvq_attn.h"
#include "nvq_attn_plan.h"
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

constexpr float kRefRoom = 15, kRefStart = 9;  // as in the few-rows kernel

// Workgroups of a kernel variant that a CU holds.
constexpr int chunk_wgs_per_cu(int D, int W) { return W == 8 || D == 256 ? 1 : D == 128 ? 2 : 3; }

// Two transpose reads -> the 8 keys of one element of an A operand: in each
// group of 16 lanes, lane i receives element i % 4 of the 8-byte reads of
// lanes i / 4 + 4 m, m = 0..3.
__device__ __forceinline__ half8_t tr_pair(const NVQ_LDS char* at, int second) {
  const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((NVQ_LDS v4i16_t*)at);
  const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((NVQ_LDS v4i16_t*)(at + second));
  const v8i16_t v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(half8_t, v);
}

// Codes and scales of one thread's share of a tile: 1 / P of the elements of
// one key, K and V (P = 4 with 4 waves, 8 with 8).
template <int D, int P>
struct TileRegs {
  static constexpr int kWords = D / 8 / P;                     // code dwords
  static constexpr int kScales = D / 16 / P > 1 ? D / 16 / P : 1;
  uint32_t k[kWords], v[kWords], ks[kScales], vs[kScales];
};

// A wave loads 64 / P keys of a tile, which lie in one page: its base is
// uniform, and a lane's offsets in it (key `key` of these, share `part`) never
// change.  id < 0 (no such page) reads page 0, masked later.  Shares of 32
// elements and more are pieces of 32, 32 P apart.
template <int D, int P>
__device__ __forceinline__ void load_tile(const AttnParams& p, TileRegs<D, P>& r, int id, int kvh, int off,
                                          uint32_t key, uint32_t part) {
  constexpr int kWords = TileRegs<D, P>::kWords;
  const int64_t tile = ((int64_t)max(id, 0) * p.c.H + kvh) << p.c.log_ps;
  const uint8_t* kc = p.c.k_codes + (tile + off) * (D / 2);
  const uint8_t* vc = p.c.v_codes + (tile + off) * (D / 2);
  const uint8_t* ks = p.c.k_scales + (tile + off) * (D / 16);
  const uint8_t* vs = p.c.v_scales + tile * (D / 16) + off;
  const uint32_t at = key * (D / 2), sat = key * (D / 16);
  if constexpr (kWords >= 4) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(kc + (at + 16 * part) + 16 * P * i);
      const uint4 y = *reinterpret_cast<const uint4*>(vc + (at + 16 * part) + 16 * P * i);
      r.k[4 * i] = x.x, r.k[4 * i + 1] = x.y, r.k[4 * i + 2] = x.z, r.k[4 * i + 3] = x.w;
      r.v[4 * i] = y.x, r.v[4 * i + 1] = y.y, r.v[4 * i + 2] = y.z, r.v[4 * i + 3] = y.w;
      const uint32_t two = *reinterpret_cast<const uint16_t*>(ks + (sat + 2 * part) + 2 * P * i);
      r.ks[2 * i] = two, r.ks[2 * i + 1] = two >> 8;
      r.vs[2 * i] = vs[key + ((2 * P * i + 2 * part) << p.c.log_ps)];
      r.vs[2 * i + 1] = vs[key + ((2 * P * i + 2 * part + 1) << p.c.log_ps)];
    }
  } else {
    if constexpr (kWords == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(kc + (at + 8 * part));
      const uint2 y = *reinterpret_cast<const uint2*>(vc + (at + 8 * part));
      r.k[0] = x.x, r.k[1] = x.y, r.v[0] = y.x, r.v[1] = y.y;
    } else {
      r.k[0] = *reinterpret_cast<const uint32_t*>(kc + (at + 4 * part));
      r.v[0] = *reinterpret_cast<const uint32_t*>(vc + (at + 4 * part));
    }
    const uint32_t blk = kWords == 2 ? part : part >> 1;
    r.ks[0] = ks[sat + blk];
    r.vs[0] = vs[key + (blk << p.c.log_ps)];
  }
}

// Byte of an E4M3 scale -> fp16 pair s_b * 2^-8, finite for any byte.
__device__ __forceinline__ uint32_t scale_of(uint32_t byte) { return (byte & 0x7Fu) * 0x00800080u; }

// Dequantizes and writes to the LDS tiles.
template <int D, int P>
__device__ __forceinline__ void store_tile(const TileRegs<D, P>& r, uint8_t* k, uint8_t* v, int part) {
  constexpr int kWords = TileRegs<D, P>::kWords, kPiece = kWords < 4 ? kWords : 4;
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    const int at = 16 * (kPiece * (P * (j / kPiece) + part) + j % kPiece);
    *reinterpret_cast<half8_t*>(k + at) = dequant8(r.k[j], scale_of(r.ks[j >> 1]));
    *reinterpret_cast<half8_t*>(v + at) = dequant8(r.v[j], scale_of(r.vs[j >> 1]));
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

// o *= keep.  With one wave per SIMD (kInAgprs) the sums live in accumulation
// registers, and are multiplied there one by one.  Written as a plain product
// the two ways out of the rare branch met in vector registers, and every tile
// moved the sums over and back (12 chunks of 700 rows at head dimension 256:
// 324 -> 299 us).  The s_nops, tied to the sums, are the wait states between
// the matrix unit's accesses to these registers and those of the vector unit.
template <bool kInAgprs, int kN>
__device__ __forceinline__ void rescale(floatx16_t (&o)[kN], float keep) {
  if constexpr (!kInAgprs) {
#pragma unroll
    for (int i = 0; i < kN; ++i) o[i] *= keep;
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      asm volatile("s_nop 15\n\ts_nop 7" : "+a"(o[i]));
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        float x = o[i][v], t;
        asm volatile("v_accvgpr_read_b32 %1, %0\n\tv_mul_f32 %1, %1, %2\n\tv_accvgpr_write_b32 %0, %1"
                     : "+a"(x), "=&v"(t)
                     : "v"(keep));
        o[i][v] = x;
      }
      asm volatile("s_nop 7" : "+a"(o[i]));
    }
  }
}

// Largest of three (v_max3_f32; fmaxf would first quiet each operand).  The
// compiler does not look into it: where b and c come out of the matrix unit, `a`
// has to depend on an ordinary operation on the same sums, before which it puts
// the wait states that such a read needs.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(m) : "v"(a), "v"(b), "v"(c));
  return m;
}

template <int D, int W>
__global__ __launch_bounds__(64 * W, chunk_wgs_per_cu(D, W) * W / 4) void k_attn_chunk(AttnParams p, ChunkPlan plan) {
  using Lds = ChunkLds<D>;
  constexpr int kSteps = D / 16, kOut = D / 32, kTileRows = 32 * W;
  __shared__ Lds lds;
  if (plan.check && blockIdx.x == 0) {
    static_assert(sizeof(CheckLds) <= sizeof(Lds));
    check_batch<64 * W>(p, reinterpret_cast<CheckLds&>(lds));
    return;
  }
  const int block = blockIdx.x - plan.check, kvh = block % p.c.H, run = block / p.c.H;
  if (run >= plan.info[0]) return;
  const bool divide = plan.info[1] != 0;
  int tile = run;
  int64_t x, x_end;
  if (divide) {
    tile = __builtin_amdgcn_readfirstlane(plan.run_tile[run]);
    x = run * plan.info[2] / plan.info[0], x_end = (run + 1) * plan.info[2] / plan.info[0];
  } else {
    x = tile ? plan.unit_end[tile - 1] : 0, x_end = plan.unit_end[tile];
  }
  const int64_t x_begin = x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float v_st = *p.c.v_st, k_factor = p.scale_log2 * *p.c.k_st;

#pragma unroll 1
  for (; x < x_end; ++tile) {
    // made anew for each tile, as in the few-rows kernel
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int l32 = lane & 31, h = lane >> 5;
    const int b = __builtin_amdgcn_readfirstlane(plan.tile[tile].x), qt = __builtin_amdgcn_readfirstlane(plan.tile[tile].y);
    const Seq s = load_seq(p, b);
    const TileRange range = tile_range(p, s, qt, kTileRows);
    const int64_t tile_x = plan.unit_end[tile] - range.units;  // its first unit
    const int u_begin = (int)(x - tile_x), u_end = (int)min<int64_t>(range.units, x_end - tile_x);
    // slot 0: the part that starts a run; 1: one that ends it and began within
    const bool whole = u_begin == 0 && u_end == range.units;
    const int64_t slot = 2 * (int64_t)run + (x != x_begin);
    x = tile_x + u_end;
    const int32_t* table = p.table + b * p.table_ld;

    // this lane's query row
    const int64_t rows = (int64_t)s.n * p.g, r = (int64_t)qt * kTileRows + 32 * wave + l32;
    const bool live = r >= 0 && r < rows;
    const int qi = live ? (int)(r / p.g) : 0, qh = kvh * p.g + (live ? (int)(r % p.g) : 0);
    // Loader: a wave takes 64 / W keys of the tile, a thread 1 / W of one of
    // them, the 16 lanes of an LDS access keys 4 apart.  Page ids of the wave's
    // next 64 tiles with one load (-1: no key, or an id outside the cache).
    const int part = lane & (W - 1);
    const int key = W == 4 ? 4 * ((lane >> 2) & 3) + (lane >> 4) : 4 * ((lane >> 3) & 1) + (lane >> 4);
    const int lkey_at = Lds::at(64 / W * wave + key);
    const int64_t base = range.base + 64 / W * wave;
    int ids = -1, ids_at = u_begin;
    auto fetch_ids = [&](int u0) {
      const int64_t first = base + (int64_t)(u0 + lane) * kTileKeys;
      const int id = (u0 + lane < u_end && first < range.hi) ? table[first >> p.c.log_ps] : -1;
      ids = id < p.c.num_pages ? id : -1;
      ids_at = u0;
    };
    TileRegs<D, W> regs;
    int id;
    auto fetch = [&](int u) {  // past the last tile: page 0, never looked at
      if (u - ids_at >= 64) fetch_ids(u);
      id = __builtin_amdgcn_readlane(ids, u - ids_at);
      load_tile<D, W>(p, regs, id, kvh, (int)(base + (int64_t)u * kTileKeys) & (p.c.ps - 1), key, part);
    };
    auto put = [&](int buf) {
      store_tile<D, W>(regs, lds.k[buf] + lkey_at, lds.v[buf] + lkey_at, part);
      if (lane == 0 && wave % (W / 4) == 0) lds.dead[buf][wave / (W / 4)] = id < 0;
    };
    // The first loads go out before any of them is waited for: page ids, the
    // query row, and the codes of the first tile.
    fetch_ids(u_begin);
    uint32_t qw[kSteps][4];
    {
      const uint16_t* at = p.q + (s.row0 + qi) * p.q_ld_t + qh * p.q_ld_h + 8 * h;
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        const uint4 x = *reinterpret_cast<const uint4*>(at + 16 * u);
        qw[u][0] = x.x, qw[u][1] = x.y, qw[u][2] = x.z, qw[u][3] = x.w;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    fetch(u_begin);
    __builtin_amdgcn_sched_barrier(0);

    half8_t qf[kSteps];
    float cq;
    {
      uint32_t top = 0;
#pragma unroll
      for (int u = 0; u < kSteps; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(qw[u][j] << 16 & 0x7FFF0000u, qw[u][j] & 0x7FFF0000u));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
      // as in the few-rows kernel; the sign of the factor goes into Q, so that
      // the largest product is the largest score, and a factor of 0 too
      const int ex = (int)(top >> 23);
      const int shift = (top == 0u || ex == 255) ? 0 : 14 + 127 - max(ex, 1);
      const float c0 = __builtin_ldexpf(k_factor, -shift);
      const float sign = c0 < 0.0f ? -1.0f : c0 > 0.0f ? 1.0f : 0.0f;
      cq = c0 == 0.0f ? 1.0f : fabsf(c0);
#pragma unroll
      for (int u = 0; u < kSteps; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qf[u][2 * j] = (_Float16)(__builtin_ldexpf(bf16_lo(qw[u][j]), shift) * sign);
          qf[u][2 * j + 1] = (_Float16)(__builtin_ldexpf(bf16_hi(qw[u][j]), shift) * sign);
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
      // Operands of the next two steps are read before the products of these:
      // left alone the compiler puts each read right before its product and
      // waits for it.
      half8_t kf[2][4];
      auto read_k = [&](half8_t (&f)[4], int w) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f[i] = *reinterpret_cast<const half8_t*>(k_at + 8 * (i & 1) * Lds::kRow + 32 * (w + (i >> 1)));
      };
      read_k(kf[0], 0);
#pragma unroll
      for (int w = 0; w < kSteps; w += 2) {
        if (w + 2 < kSteps) read_k(kf[(w >> 1 & 1) ^ 1], w + 2);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i)  // two chains of products in turn
          sc[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[w >> 1 & 1][i], qf[w + (i >> 1)], sc[i & 1], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
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
      const float first = fmaxf(sc[0][0], sc[1][0]);
      float top = max3(first, sc[0][1], sc[1][1]), top2 = max3(first, sc[0][2], sc[1][2]);
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
        rescale<D == 256>(o, keep);
      }
      const NVQ_LDS char* vt = (const NVQ_LDS char*)lds.v[buf] + tr_off;
      half8_t vf[2][kOut], pf[2];
      auto read_v = [&](half8_t (&f)[kOut], int j) {
#pragma unroll
        for (int i = 0; i < kOut; ++i) f[i] = tr_pair(vt + 4 * j * Lds::kRow + 64 * i, 2 * Lds::kRow);
      };
      auto weights = [&](half8_t& f, int j) {  // of 16 keys
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[j >> 1][8 * (j & 1) + v], cq, -ref_safe));
          l += w;
          f[v] = (_Float16)w;
        }
      };
      read_v(vf[0], 0);
      weights(pf[0], 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < 3) read_v(vf[(j & 1) ^ 1], j + 1);
        if (j < 3)
          weights(pf[(j & 1) ^ 1], j + 1);
        else
          put(buf ^ 1);
#pragma unroll
        for (int i = 0; i < kOut; ++i)
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[j & 1][i], pf[j & 1], o[i], 0, 0, 0);
      }
      __syncthreads();
    }

    l += __shfl_xor(l, 32, 64);
    if (whole) {
      if (live) {
        const OutScale scale(l, v_st);
        uint16_t* out = p.out + (s.row0 + qi) * p.out_ld_t + qh * p.out_ld_h;
#pragma unroll
        for (int i = 0; i < kOut; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            *reinterpret_cast<uint2*>(out + 32 * i + 8 * v + 4 * h) =
                make_uint2(scale.bf16(o[i][4 * v]) | (scale.bf16(o[i][4 * v + 1]) << 16),
                           scale.bf16(o[i][4 * v + 2]) | (scale.bf16(o[i][4 * v + 3]) << 16));
        if (p.lse && h == 0)
          p.lse[(int64_t)(s.row0 + qi) * p.Hq + qh] = l == 0.0f ? -INFINITY : (ref + __builtin_log2f(l)) * kLn2;
      }
    } else {
      const int64_t at = (slot * p.c.H + kvh) * kTileRows + 32 * wave + l32;
      float* out = plan.part_o + at * D;
#pragma unroll
      for (int i = 0; i < kOut; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          *reinterpret_cast<float4*>(out + 32 * i + 8 * v + 4 * h) =
              make_float4(o[i][4 * v], o[i][4 * v + 1], o[i][4 * v + 2], o[i][4 * v + 3]);
      if (h == 0) plan.part_ml[at] = make_float2(ref, l);
    }
  }
}

template <int D, int W>
int launch_chunk(const AttnParams& p, const ChunkPlan& plan, hipStream_t s) {
  const int64_t runs = std::max<int64_t>(plan.max_tiles, plan.workers);
  hipLaunchKernelGGL((k_attn_chunk<D, W>), dim3((unsigned)(runs * p.c.H + plan.check)), dim3(64 * W), 0, s, p, plan);
  return last_launch();
}

__global__ __launch_bounds__(1024) void k_attn_chunk_plan(AttnParams p, ChunkPlan plan) {
  __shared__ PlanLds lds;
  plan_chunks(p, plan, lds);
}

}  // namespace

void attn_chunk_plan(const AttnParams& p, int min_rows, bool check, WsCarve& ws, ChunkPlan& plan) {
  plan.min_rows = min_rows;
  plan.check = check;
  // Head dimension 128: 256-row tiles halve the dequantization of a row, but
  // only one workgroup fits a CU, so nothing covers the start and the end of a
  // tile; two with 128 rows where rows see few keys.  32 heads on 8: chunks of
  // 1024 and 1536 new tokens 71 us against 81 and 93 against 107, windows of 512
  // and 1024 129 against 147 and 192 against 203; two chunks of 2048 96 against
  // 104, 4096 behind 4096 713 against 741.
  const bool far = p.window > 0 ? std::min(p.window, p.num_keys) > 1024 : p.num_keys >= 2048;
  const int waves = p.c.D == 128 && (int64_t)p.max_q * p.g > 128 && far ? 8 : 4;
  plan.tile_rows = 32 * waves;
  // rows of a sequence are cut to the call's, so its tiles are at most this
  plan.max_tiles = (int64_t)p.total_q * p.g / plan.tile_rows + p.B;
  const int64_t units = (p.num_keys + kTileKeys - 1) / kTileKeys + 1;  // most of a tile
  plan.per_cu = chunk_wgs_per_cu(p.c.D, waves);
  const int64_t places = (int64_t)plan.per_cu * device_cu_count() - plan.check;
  plan.places = (int)std::max<int64_t>(1, places / p.c.H);
  plan.workers = (int)std::max<int64_t>(1, std::min<int64_t>(plan.places, units * plan.max_tiles / kChunkMinUnits));
  plan.info = ws.take<int64_t>(3);
  plan.tile_end = ws.take<int32_t>((size_t)p.B);
  plan.tile = ws.take<int2>((size_t)plan.max_tiles);
  plan.unit_end = ws.take<int64_t>((size_t)plan.max_tiles);
  plan.run_tile = ws.take<int32_t>((size_t)plan.workers);
  const size_t rows = plan.workers > 1 ? (size_t)(2 * plan.workers * p.c.H) * plan.tile_rows : 0;
  plan.part_ml = ws.take<float2>(rows);
  plan.part_o = ws.take<float>(rows * p.c.D);
}

int attn_chunk_launch(const AttnParams& p, const ChunkPlan& plan, bool planned, hipStream_t s) {
  if (!planned) {
    hipLaunchKernelGGL(k_attn_chunk_plan, dim3(1), dim3(1024), 0, s, p, plan);
    if (int rc = last_launch()) return rc;
  }
  switch (p.c.D * 16 + plan.tile_rows / 32) {
    case 64 * 16 + 4: return launch_chunk<64, 4>(p, plan, s);
    case 128 * 16 + 4: return launch_chunk<128, 4>(p, plan, s);
    case 128 * 16 + 8: return launch_chunk<128, 8>(p, plan, s);
    default: return launch_chunk<256, 4>(p, plan, s);
  }
}

}  // namespace nvq
