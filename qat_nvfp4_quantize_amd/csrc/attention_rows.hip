// Attention over the paged NVFP4 cache for sequences of few query rows per
// key/value head (single tokens, drafts): HBM-bound, the cache's 0.5625 bytes
// a value are read once and little is done with each.
//
// A wave takes 32 keys at a time straight from memory into MFMA operands: no
// LDS on the way.  Both products run transposed, S^T = K Q^T and O^T = V^T P^T
// (16x16x32 fp16), so that a lane always holds one query (column) and several
// keys or elements (rows):
//  * K: lane (key n, group q) loads the codes of D / 4 consecutive elements,
//    q D/4 .., of its key; MFMA step w takes its w-th eight.  Any order of
//    the contraction works because Q is held in the same one.
//  * S^T leaves lane (query n, q) the keys 16 t + 4 q + v: softmax needs no
//    lane exchange, and its weights are already the B operand of O^T with the
//    contraction order (t, v) per lane.
//  * V: lane (n, q) loads, for those 8 keys, the codes of elements n D/16 ..
//    n D/16 + D/16 - 1; tile u of O^T takes the u-th of them, so a byte
//    permute pairs the keys of an element and one packed multiply applies two
//    block scales (one dword holds the scales of four consecutive slots).
// The reference of the running softmax is only moved when a score exceeds it
// by 15 (in powers of two): weights stay within fp16, and a step without a
// move rescales nothing.  Weights are rounded to fp16 because that is the matrix
// unit's operand (bf16 would keep three bits less); their sum takes them as
// they were.  Each is off by 2^-11 of itself at most, an eighth of half a step of
// the bf16 result: outputs lie as far from 64 bits as rounding alone puts them
// (relative rms 0.0016 to 0.0018, 0.0016 to 0.0017 with fp32 weights), about one
// in ten on the neighbouring bf16 value.
//
// Work is split over the keys: per key/value head, the units of all sequences
// in one row are dealt to as many workers as the chip holds at once, in equal
// runs, whatever the lengths (every wave finds its run from cu_q and kv_len
// itself).  A worker is a workgroup, each of its four waves taking 32 keys of a
// 128-key unit, or (W = 1), where there are many sequences, a wave with units
// of 32: no exchange between waves, a quarter of the set-up of a sequence, but
// four times the runs, hence more parts.  A run may end inside a sequence: the
// parts of such sequences are joined by a second kernel.  Equal runs matter:
// with pieces cut per sequence 64 ragged sequences made 1232 pieces for 768
// places, two rounds of 33 us.
//
// Measured: 64 sequences of up to 8192 keys, 32 heads on 8 of 128: 72 us (a
// copy moves the same bytes in 63), of which the loop takes 57 at 5.6 TB/s, the
// rest goes to finding the runs, the first loads and the join; one sequence of
// 131072 keys, 64 heads on 8: 43 us (30).

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

typedef float floatx4_t __attribute__((ext_vector_type(4)));

// Keys of a step: 32 of each of a worker's W waves.
constexpr int unit_keys(int W) { return 32 * W; }
constexpr float kRefRoom = 15;  // a score may exceed the reference by this (2^15 < fp16's largest)
constexpr float kRefStart = 9;  // and the reference is set this much below the largest score seen

// Keys [lo, hi) that some row of sequence s sees, in 32-key steps from `base`.
struct Range {
  int64_t base, hi;
  int units;
};
template <int W>
__device__ __forceinline__ Range key_range(const AttnParams& p, const Seq& s) {
  constexpr int kUnit = unit_keys(W);
  Range r;
  int64_t lo, x;
  visible(p, s, s.pos0, lo, x);
  visible(p, s, s.pos0 + s.n - 1, x, r.hi);
  r.base = lo & ~(int64_t)31;
  r.units = r.hi > r.base ? (int)((r.hi - r.base + kUnit - 1) / kUnit) : 1;
  return r;
}

// Units up to and with sequence 64 c + lane, within its chunk of 64.
template <int W>
__device__ __forceinline__ int chunk_units(const AttnParams& p, int max_rows, int c) {
  const int b = 64 * c + (threadIdx.x & 63);
  int units = 0;
  if (b < p.B) {
    const Seq s = load_seq(p, b);
    if (s.n > 0 && s.n * p.g <= max_rows) units = key_range<W>(p, s).units;
  }
  return wave_inclusive_scan(units);
}

// Units of a workgroup's run, where there are so many; and most units of a
// sequence that takes one workgroup a head whole, which spares the joining
// launch (one of 777 keys: 13.1 us against 15.4, of 1024: 14.2 against 15.4, of
// 1500: 17.7 against 14.8; 60 of up to 900: 16.6 against 21.1, 24 of up to 459:
// 11.6 against 14.9).
constexpr int kMinUnits = 2, kFewUnits = 9;

// Workgroups of a kernel variant that a CU holds (its register budget).
constexpr int rows_wgs_per_cu(int D, int MT) {
  return D * MT <= 64 ? 4 : D * MT <= 128 ? 3 : D * MT <= 256 ? 2 : 1;
}

// Codes and scales of one wave step (32 keys) in registers.
template <int D>
struct StepRegs {
  static constexpr int kKW = D / 32;                  // dwords of K codes of a lane and half
  static constexpr int kVW = D / 128 > 1 ? D / 128 : 1;  // dwords of V codes of a lane and key
  uint32_t k[2][kKW], ks[2], v[8][kVW], vs[2];
};

// Bases are wave-uniform (the page ids come from a readlane) and a lane's
// offsets inside a 16-key group never change, so the loads need no address
// arithmetic in vector registers.
template <int D>
__device__ __forceinline__ void load_step(const AttnParams& p, StepRegs<D>& r, const int (&id)[2], int kvh, int off0,
                                          int lane) {
  const uint32_t n = lane & 15, q = lane >> 4;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int64_t tile = ((int64_t)max(id[t], 0) * p.c.H + kvh) << p.c.log_ps;  // a masked page reads page 0
    const int off = (off0 + 16 * t) & (p.c.ps - 1);
    const uint8_t* kc = p.c.k_codes + (tile + off) * (D / 2);
    const uint32_t kl = n * (D / 2) + q * (D / 8);
    if constexpr (D == 64) {
      const uint2 w = *reinterpret_cast<const uint2*>(kc + kl);
      r.k[t][0] = w.x, r.k[t][1] = w.y;
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(kc + kl + 16 * i);
        r.k[t][4 * i] = w.x, r.k[t][4 * i + 1] = w.y, r.k[t][4 * i + 2] = w.z, r.k[t][4 * i + 3] = w.w;
      }
    }
    const uint8_t* ks = p.c.k_scales + (tile + off) * (D / 16);
    const uint32_t sl = n * (D / 16) + q * (D / 64);
    if constexpr (D == 64)
      r.ks[t] = ks[sl];
    else if constexpr (D == 128)
      r.ks[t] = *reinterpret_cast<const uint16_t*>(ks + sl);
    else
      r.ks[t] = *reinterpret_cast<const uint32_t*>(ks + sl);
    const uint8_t* vc = p.c.v_codes + (tile + off) * (D / 2);
    const uint32_t vl = 4 * q * (D / 2) + n * (D / 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t(&w)[StepRegs<D>::kVW] = r.v[4 * t + i];
      if constexpr (D == 64) {
        w[0] = *reinterpret_cast<const uint16_t*>(vc + vl + i * (D / 2));
      } else if constexpr (D == 128) {
        w[0] = *reinterpret_cast<const uint32_t*>(vc + vl + i * (D / 2));
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(vc + vl + i * (D / 2));
        w[0] = x.x, w[1] = x.y;
      }
    }
    const uint8_t* vs = p.c.v_scales + tile * (D / 16) + off;
    r.vs[t] = *reinterpret_cast<const uint32_t*>(vs + ((n * D / 256) << p.c.log_ps) + 4 * q);
  }
}

template <int kSel>
__device__ __forceinline__ uint32_t fp4_pair_f16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, kSel));
}

// Two elements (byte kSel of each key's codes) of 8 keys -> the A operands of
// two tiles: element e of keys 0..7 times the keys' block scales.
template <int kSel>
__device__ __forceinline__ void v_operands(const uint32_t (&w)[8], const half2_t (&sc)[4], half8_t& lo, half8_t& hi) {
  uint32_t a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t e0 = fp4_pair_f16<kSel>(w[2 * i]), e1 = fp4_pair_f16<kSel>(w[2 * i + 1]);
    const half2_t x = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(e1, e0, 0x05040100u)) * sc[i];
    const half2_t y = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(e1, e0, 0x07060302u)) * sc[i];
    a[i] = __builtin_bit_cast(uint32_t, x);
    b[i] = __builtin_bit_cast(uint32_t, y);
  }
  __builtin_memcpy(&lo, a, 16);
  __builtin_memcpy(&hi, b, 16);
}

// Bytes 2 i, 2 i + 1 of a dword of E4M3 scales -> fp16 pair s_b * 2^-8.
__device__ __forceinline__ half2_t scale_two(uint32_t four, int i) {
  return __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0u, four, i ? 0x0C030C02u : 0x0C010C00u) << 7);
}

template <int D, int MT, int W>
__global__ __launch_bounds__(256, rows_wgs_per_cu(D, MT)) void k_attn_rows(AttnParams p, RowsPlan plan,
                                                                           ChunkPlan chunks) {
  constexpr int kRows = 16 * MT, kTiles = D / 16, kSteps = D / 32, kUnit = unit_keys(W);
  constexpr int kPitch = D + 4;  // floats; 16-byte rows shifted over the banks
  __shared__ float s_o[2][kRows * kPitch];
  __shared__ float s_m[4][kRows], s_l[4][kRows];
  __shared__ union {
    CheckLds check;
    PlanLds plan;
  } s_one;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // one workgroup more than workers, and one that plans the many-rows launch
  if (blockIdx.x == 0) {
    check_batch<256>(p, s_one.check);
    return;
  }
  if (plan.plans_chunks && blockIdx.x == 1) {
    plan_chunks(p, chunks, s_one.plan);
    return;
  }
  const int block = blockIdx.x - 1 - plan.plans_chunks, kvh = block % p.c.H;
  const int worker = W == 4 ? block / p.c.H : block / p.c.H * 4 + wave, share = W == 4 ? wave : 0;  // share of a unit

  // this worker's run [x, x_end) of the units of all sequences
  int chunk = W == 4 && plan.whole ? worker >> 6 : 0;
  int incl = chunk_units<W>(p, plan.max_rows, chunk), total = __builtin_amdgcn_readlane(incl, 63), workers = 1;
  int x, x_end;
  if (W == 4 && plan.whole) {  // a sequence
    x = (worker & 63) ? __builtin_amdgcn_readlane(incl, (worker & 63) - 1) : 0;
    x_end = __builtin_amdgcn_readlane(incl, worker & 63);
  } else {
    for (int c = 1; 64 * c < p.B; ++c) total += __builtin_amdgcn_readlane(chunk_units<W>(p, plan.max_rows, c), 63);
    workers = min(plan.workers, max(1, total / (kMinUnits * 4 / W)));
    if (worker >= workers) return;
    x = (int)((int64_t)worker * total / workers);
    x_end = (int)((int64_t)(worker + 1) * total / workers);
  }
  if (x == x_end) return;
  const int x_begin = x;
  int before = 0;  // units of earlier chunks
  const float c0 = p.scale_log2 * *p.c.k_st, v_st = *p.c.v_st;

#pragma unroll 1
  while (x < x_end) {
    // Made anew for each sequence: what the compiler would otherwise carry
    // over from one to the next in registers ends in scratch memory, whose
    // loads then wait in line with the cache's.
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int n = lane & 15, q = lane >> 4;
    // the sequence of unit x, and the units of it in this run
    uint64_t past = __ballot(before + incl > x);
    while (!past) {
      if (64 * (chunk + 1) >= p.B) return;  // only if the arrays change under the call
      before += __builtin_amdgcn_readlane(incl, 63);
      incl = chunk_units<W>(p, plan.max_rows, ++chunk);
      past = __ballot(before + incl > x);
    }
    const int sl = __builtin_ctzll(past), b = 64 * chunk + sl;
    const Seq s = load_seq(p, b);
    const Range range = key_range<W>(p, s);
    const int seq_x = before + __builtin_amdgcn_readlane(incl, sl) - range.units;  // its first unit
    const int u_begin = x - seq_x, u_end = min(range.units, x_end - seq_x);
    // a part that starts a run goes to the worker's slot 0, one that ends it
    // inside a sequence begun within the run to slot 1
    const bool whole_seq = u_begin == 0 && u_end == range.units;
    const int slot = x == x_begin ? 2 * worker : 2 * worker + 1;
    if (plan.may_split && u_begin == 0 && kvh == 0 && (W == 4 ? threadIdx.x : threadIdx.x & 63) == 0) {
      const int last = (int)(((int64_t)(seq_x + range.units) * workers - 1) / total);
      plan.seq[2 * b] = slot;
      plan.seq[2 * b + 1] = last - worker + 1;
    }
    if (W == 4 && x != x_begin) __syncthreads();  // the last sequence's LDS reads are done
    x = seq_x + u_end;
    const int rows = s.n * p.g;
    const int32_t* table = p.table + b * p.table_ld;

    // Page ids of the wave's next 32 steps, one load: lane 2 i + t has those of
    // step i's half t (-1: no key, or an id outside the cache).
    int ids = -1, ids_at = u_begin;
    auto fetch_ids = [&](int u0) {
      const int64_t key = range.base + (int64_t)(u0 + (lane >> 1)) * kUnit + 32 * share + 16 * (lane & 1);
      int id = key < range.hi ? table[key >> p.c.log_ps] : -1;
      if (id >= p.c.num_pages) id = -1;
      ids = id;
      ids_at = u0;
    };
    auto page_pair = [&](int u, int (&id)[2]) {
      if (u - ids_at >= 32) fetch_ids(u);
      id[0] = __builtin_amdgcn_readlane(ids, 2 * (u - ids_at));
      id[1] = __builtin_amdgcn_readlane(ids, 2 * (u - ids_at) + 1);
    };

    const int64_t base = range.base + 32 * share;
    auto fetch = [&](StepRegs<D>& regs, int (&id)[2], int u) {
      page_pair(u, id);
      load_step<D>(p, regs, id, kvh, (int)((base + (int64_t)u * kUnit) & (p.c.ps - 1)), lane);
    };
    // The first loads go out before any of them is waited for: page ids, the
    // query rows, and the codes of the first step.
    fetch_ids(u_begin);
    uint32_t qw[MT][kSteps][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = 16 * mt + n, i = r < rows ? r / p.g : 0, h = kvh * p.g + (r < rows ? r - i * p.g : 0);
      const uint16_t* at = p.q + (s.row0 + i) * p.q_ld_t + h * p.q_ld_h + q * (D / 4);
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        const uint4 x = *reinterpret_cast<const uint4*>(at + 8 * u);
        qw[mt][u][0] = x.x, qw[mt][u][1] = x.y, qw[mt][u][2] = x.z, qw[mt][u][3] = x.w;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    StepRegs<D> cur, nxt;
    int id_cur[2], id_nxt[2];
    fetch(cur, id_cur, u_begin);
    __builtin_amdgcn_sched_barrier(0);

    // Q in fp16 under a power of two per row that brings its largest magnitude
    // to 2^14 .. 2^15: all 8 bits of bf16 are kept down to 2^-31 of it (steps of
    // 2^-24 below 2^-14 in fp16), and no element is off by more than 2^-39 of it.
    half8_t qf[MT][kSteps];
    float cq[MT];
    int see_lo[MT], see_hi[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = 16 * mt + n;
      const bool live = r < rows;
      uint32_t(&w)[kSteps][4] = qw[mt];
      uint32_t top = 0;
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[u][j] = live ? w[u][j] : 0u;
          top = max(top, max(w[u][j] << 16 & 0x7FFF0000u, w[u][j] & 0x7FFF0000u));
        }
      }
      top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
      const int ex = (int)(top >> 23);
      const int shift = (top == 0u || ex == 255) ? 0 : 14 + 127 - max(ex, 1);
#pragma unroll
      for (int u = 0; u < kSteps; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qf[mt][u][2 * j] = (_Float16)__builtin_ldexpf(bf16_lo(w[u][j]), shift);
          qf[mt][u][2 * j + 1] = (_Float16)__builtin_ldexpf(bf16_hi(w[u][j]), shift);
        }
      cq[mt] = __builtin_ldexpf(c0, -shift);
      int64_t lo, hi;
      visible(p, s, s.pos0 + r / p.g, lo, hi);
      see_lo[mt] = (int)min<int64_t>(lo, INT32_MAX);
      see_hi[mt] = live ? (int)max<int64_t>(hi, 0) : 0;
    }
    // every row sees all of [all_lo, all_hi)
    int64_t all_lo, all_hi, x64;
    visible(p, s, s.pos0, x64, all_hi);
    visible(p, s, s.pos0 + s.n - 1, all_lo, x64);

    floatx4_t o[MT][kTiles];
    float ref[MT], ref_safe[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      ref[mt] = -INFINITY, ref_safe[mt] = 0.0f, l[mt] = 0.0f;
#pragma unroll
      for (int u = 0; u < kTiles; ++u) o[mt][u] = (floatx4_t)(0.0f);
    }

    auto consume = [&](const StepRegs<D>& cur, const int (&id)[2], int u) {
      const int64_t kb = base + (int64_t)u * kUnit;
      if (kb < range.hi) {
        floatx4_t sc[MT][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t ks = cur.ks[t] & 0x7F7F7F7Fu;  // finite for any byte
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) sc[mt][t] = (floatx4_t)(0.0f);
#pragma unroll
          for (int w = 0; w < kSteps; ++w) {
            const half8_t a = dequant8(cur.k[t][w], scale_pair(ks, w >> 1));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              sc[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, qf[mt][w], sc[mt][t], 0, 0, 0);
          }
        }
        const bool whole = kb >= all_lo && kb + 32 <= all_hi && id[0] >= 0 && id[1] >= 0;
        half8_t pf[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float top = -INFINITY;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float x = sc[mt][t][v] * cq[mt];
              if (!whole) {
                const int key = (int)kb + 16 * t + 4 * q + v;
                x = (key >= see_lo[mt] && key < see_hi[mt] && id[t] >= 0) ? x : -INFINITY;
              }
              sc[mt][t][v] = x;
              top = fmaxf(top, x);
            }
          if (__ballot(top > ref[mt] + kRefRoom)) {
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float moved = top > ref[mt] + kRefRoom ? top - kRefStart : ref[mt];
            const float keep = moved == ref[mt] ? 1.0f : __builtin_amdgcn_exp2f(ref[mt] - moved);
            ref[mt] = moved;
            ref_safe[mt] = moved == -INFINITY ? 0.0f : moved;
            l[mt] *= keep;
#pragma unroll
            for (int i = 0; i < kTiles; ++i) o[mt][i] *= keep;
          }
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const float w = __builtin_amdgcn_exp2f(sc[mt][t][v] - ref_safe[mt]);
              l[mt] += w;
              pf[mt][4 * t + v] = (_Float16)w;
            }
        }
        half2_t vs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) vs[i] = scale_two(cur.vs[i >> 1] & 0x7F7F7F7Fu, i & 1);
#pragma unroll
        for (int j = 0; j < StepRegs<D>::kVW; ++j) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = cur.v[i][j];
          half8_t a[8];
          v_operands<0>(w, vs, a[0], a[1]);
          v_operands<1>(w, vs, a[2], a[3]);
          if constexpr (D > 64) {
            v_operands<2>(w, vs, a[4], a[5]);
            v_operands<3>(w, vs, a[6], a[7]);
          }
#pragma unroll
          for (int e = 0; e < (D > 64 ? 8 : 4); ++e)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              o[mt][8 * j + e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[e], pf[mt], o[mt][8 * j + e], 0, 0, 0);
        }
      }
    };
#pragma unroll 1
    for (int u = u_begin; u < u_end; ++u) {  // the next step's loads are in flight while a step is computed
      if (u + 1 < u_end) fetch(nxt, id_nxt, u + 1);
      consume(cur, id_cur, u);
      cur = nxt;
      id_cur[0] = id_nxt[0], id_cur[1] = id_nxt[1];
    }

    if constexpr (W == 4) {
      // Join the four waves: each scales its part to the common reference, waves
      // 2 and 3 hand theirs over through LDS, waves 0 and 1 add and leave two
      // parts for the workgroup.
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        l[mt] += __shfl_xor(l[mt], 16, 64);
        l[mt] += __shfl_xor(l[mt], 32, 64);
        if (q == 0) s_m[wave][16 * mt + n] = ref[mt], s_l[wave][16 * mt + n] = l[mt];
      }
      __syncthreads();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int r = 16 * mt + n;
        const float m = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
        const float f = ref[mt] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ref[mt] - m);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) o[mt][i] *= f;
      }
      float* part = s_o[wave & 1];
      auto each = [&](auto&& f) {  // float4 of 4 consecutive elements of the lane's row
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int i = 0; i < kTiles / 4; ++i)
              f(reinterpret_cast<float4*>(part + (16 * mt + n) * kPitch + (4 * q + v) * kTiles + 4 * i),
                make_float4(o[mt][4 * i][v], o[mt][4 * i + 1][v], o[mt][4 * i + 2][v], o[mt][4 * i + 3][v]));
      };
      if (wave >= 2) each([](float4* at, float4 x) { *at = x; });
      __syncthreads();
      if (wave < 2)
        each([](float4* at, float4 x) {
          const float4 y = *at;
          *at = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        });
      __syncthreads();
      constexpr int kChunks = D / 8;
      for (int e = threadIdx.x; e < kRows * kChunks; e += 256) {
        const int r = e / kChunks, ch = e - r * kChunks;
        if (r >= rows) break;
        const float m = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
        float sum = 0.0f;  // a wave whose scores are all NaN has no reference either, but a sum of NaN: it counts
#pragma unroll
        for (int w = 0; w < 4; ++w)
          sum += s_l[w][r] * (s_m[w][r] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(s_m[w][r] - m));
        float x[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 a = *reinterpret_cast<const float4*>(s_o[0] + r * kPitch + 8 * ch + 4 * i);
          const float4 b = *reinterpret_cast<const float4*>(s_o[1] + r * kPitch + 8 * ch + 4 * i);
          x[4 * i] = a.x + b.x, x[4 * i + 1] = a.y + b.y, x[4 * i + 2] = a.z + b.z, x[4 * i + 3] = a.w + b.w;
        }
        if (whole_seq) {
          const int i = r / p.g, h = kvh * p.g + (r - i * p.g);
          const OutScale scale(sum, v_st);
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = scale.bf16(x[2 * j]) | (scale.bf16(x[2 * j + 1]) << 16);
          *reinterpret_cast<uint4*>(p.out + (s.row0 + i) * p.out_ld_t + h * p.out_ld_h + 8 * ch) =
              make_uint4(w[0], w[1], w[2], w[3]);
          if (p.lse && ch == 0)
            p.lse[(int64_t)(s.row0 + i) * p.Hq + h] = sum == 0.0f ? -INFINITY : (m + __builtin_log2f(sum)) * kLn2;
        } else {
          const int64_t at_row = ((int64_t)slot * p.c.H + kvh) * plan.part_rows + r;
          float4* at = reinterpret_cast<float4*>(plan.part_o + at_row * D + 8 * ch);
          at[0] = make_float4(x[0], x[1], x[2], x[3]);
          at[1] = make_float4(x[4], x[5], x[6], x[7]);
          if (ch == 0) plan.part_ml[at_row] = make_float2(m, sum);
        }
      }
    } else {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        l[mt] += __shfl_xor(l[mt], 16, 64);
        l[mt] += __shfl_xor(l[mt], 32, 64);
        const int r = 16 * mt + n;
        if (r >= rows) continue;
        if (whole_seq) {
          const int i = r / p.g, h = kvh * p.g + (r - i * p.g);
          const OutScale scale(l[mt], v_st);
          uint16_t* out = p.out + (s.row0 + i) * p.out_ld_t + h * p.out_ld_h + 4 * q * kTiles;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t w[kTiles / 2];
#pragma unroll
            for (int j = 0; j < kTiles / 2; ++j)
              w[j] = scale.bf16(o[mt][2 * j][v]) | (scale.bf16(o[mt][2 * j + 1][v]) << 16);
            __builtin_memcpy(__builtin_assume_aligned(out + v * kTiles, kTiles < 8 ? 8 : 16), w, sizeof(w));
          }
          if (p.lse && q == 0)
            p.lse[(int64_t)(s.row0 + i) * p.Hq + h] =
                l[mt] == 0.0f ? -INFINITY : (ref[mt] + __builtin_log2f(l[mt])) * kLn2;
        } else {
          const int64_t at_row = ((int64_t)slot * p.c.H + kvh) * plan.part_rows + r;
          float* at = plan.part_o + at_row * D + 4 * q * kTiles;
#pragma unroll
          for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int i = 0; i < kTiles; i += 4)
              *reinterpret_cast<float4*>(at + v * kTiles + i) =
                  make_float4(o[mt][i][v], o[mt][i + 1][v], o[mt][i + 2][v], o[mt][i + 3][v]);
          if (q == 0) plan.part_ml[at_row] = make_float2(ref[mt], l[mt]);
        }
      }
    }
  }
}

template <int D, int MT>
int launch_rows(const AttnParams& p, const RowsPlan& plan, const ChunkPlan& chunk, hipStream_t s) {
  const dim3 grid((unsigned)(plan.workers * plan.waves / 4 * p.c.H + 1 + plan.plans_chunks));
  if (plan.waves == 4)
    hipLaunchKernelGGL((k_attn_rows<D, MT, 4>), grid, dim3(256), 0, s, p, plan, chunk);
  else
    hipLaunchKernelGGL((k_attn_rows<D, MT, 1>), grid, dim3(256), 0, s, p, plan, chunk);
  return last_launch();
}

}  // namespace

// Row tiles of 16 that the kernel takes for sequences of up to `rows` rows per
// key/value head; 0: none.
int attn_rows_tiles(int D, int64_t rows) {
  return rows <= (D == 256 ? 32 : 64) ? (int)((rows + 15) / 16) : 0;
}

void attn_rows_plan(const AttnParams& p, int tiles, bool chunks, WsCarve& ws, RowsPlan& plan) {
  plan.plans_chunks = chunks;
  plan.max_rows = 16 * tiles;
  // most keys of a sequence, from a multiple of 32 on, and units
  const int64_t keys = p.window > 0 ? std::min(p.num_keys, p.window + p.max_q + 30) : p.num_keys;
  const int64_t units = std::max<int64_t>(1, (keys + unit_keys(4) - 1) / unit_keys(4));
  const int64_t places = (int64_t)rows_wgs_per_cu(p.c.D, tiles) * device_cu_count();
  plan.workers = (int)std::max<int64_t>(1, std::min((places - 1 - chunks) / p.c.H, units * p.B / kMinUnits));
  // Waves as workers from a sequence for two workgroups on, if each of these
  // would have eight units (head dimension 128, 32 heads on 8: 1024 sequences of
  // up to 512 keys 109 us against 134, 256 of 1024 53 against 57, 64 of 8192 74
  // against 75; 16 of 4000 22 against 21, 50 of 600 22 against 19).
  const bool many = plan.workers > 1 && plan.workers <= 2 * p.B && units * p.B >= 8 * plan.workers &&
                    p.B * (p.num_keys / 32 + 2) <= INT32_MAX;
  plan.waves = many ? 1 : 4;
  plan.whole = !many && units <= kFewUnits;
  plan.workers = plan.whole ? (int)p.B : plan.workers * (4 / plan.waves);
  plan.may_split = !plan.whole && plan.workers > 1;
  plan.part_rows = (int)std::min<int64_t>(plan.max_rows, ((int64_t)p.max_q * p.g + 3) / 4 * 4);  // joined by fours
  plan.seq = ws.take<int32_t>(2 * (size_t)p.B);
  const size_t rows = plan.may_split ? (size_t)(2 * plan.workers * p.c.H) * plan.part_rows : 0;
  plan.part_ml = ws.take<float2>(rows);
  plan.part_o = ws.take<float>(rows * p.c.D);
}

int attn_rows_launch(const AttnParams& p, const RowsPlan& plan, const ChunkPlan& chunk, hipStream_t s) {
  switch (p.c.D * 8 + plan.max_rows / 16) {
    case 64 * 8 + 1: return launch_rows<64, 1>(p, plan, chunk, s);
    case 64 * 8 + 2: return launch_rows<64, 2>(p, plan, chunk, s);
    case 64 * 8 + 3: return launch_rows<64, 3>(p, plan, chunk, s);
    case 64 * 8 + 4: return launch_rows<64, 4>(p, plan, chunk, s);
    case 128 * 8 + 1: return launch_rows<128, 1>(p, plan, chunk, s);
    case 128 * 8 + 2: return launch_rows<128, 2>(p, plan, chunk, s);
    case 128 * 8 + 3: return launch_rows<128, 3>(p, plan, chunk, s);
    case 128 * 8 + 4: return launch_rows<128, 4>(p, plan, chunk, s);
    case 256 * 8 + 1: return launch_rows<256, 1>(p, plan, chunk, s);
    default: return launch_rows<256, 2>(p, plan, chunk, s);
  }
}

}  // namespace nvq
