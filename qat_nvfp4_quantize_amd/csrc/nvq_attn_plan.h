// Row tiles of the many-rows attention kernel and the plan of a call: used by
// the workgroup that plans, which rides on the few-rows launch where a batch
// has one, and by the kernel itself.
#pragma once

#include <hip/hip_runtime.h>

#include "nvq_attn.h"
#include "nvq_scan.h"

namespace nvq {

constexpr int kTileKeys = 64;
constexpr int kChunkMinUnits = 2;  // key tiles of a run, at least
// Row tiles go out whole (sequences in the batch's order; within one the last
// rows, which see the most keys, first), or their units are dealt in equal runs,
// whose divided tiles leave parts that the join reads: about 4 units' time, and
// 16 more if all places take part.  With this many tiles per place they go out
// whole in any case, also where one tile is far longer than the others; with
// fewer, whichever is expected to take less: 1000 new tokens, 32 heads on 8 of
// 128, 39 us whole against 71; 79 behind 1116 of one head of 256 31 us divided
// against 60.  A workgroup alone on a CU that holds more takes kLonePace of a
// unit's time (1523 new tokens, 16 heads on 4 of 64: 46 us whole against 68).
constexpr float kWholeTiles = 1.5f, kJoinUnits = 4, kPartUnits = 16, kLonePace = 0.6f;

// Keys of row tile qt of sequence s, in 64-key tiles from `base`.
struct TileRange {
  int64_t base, hi;
  int units;
};
__device__ __forceinline__ TileRange tile_range(const AttnParams& p, const Seq& s, int qt, int tile_rows) {
  const int i0 = (int)((int64_t)qt * tile_rows / p.g);
  const int i1 = min(s.n - 1, (int)(((int64_t)(qt + 1) * tile_rows - 1) / p.g));
  TileRange r;
  int64_t lo, x;
  visible(p, s, s.pos0 + i0, lo, x);
  visible(p, s, s.pos0 + i1, x, r.hi);
  r.base = lo & ~(int64_t)(kTileKeys - 1);
  r.units = r.hi > r.base ? (int)((r.hi - r.base + kTileKeys - 1) / kTileKeys) : 1;
  return r;
}

struct PlanLds {
  int end[1024];  // tile_end of the first 1024 sequences
  int scan[16];
  int64_t last;
};

// One workgroup (256 or 1024 threads) plans the call: the row tiles of the
// sequences (the last rows, which see the most keys, first), the units up to
// each, and the cuts.  Row ranges that overlap could name more tiles than the
// buffers hold: the count is cut there.
__device__ __forceinline__ void plan_chunks(const AttnParams& p, const ChunkPlan& plan, PlanLds& lds) {
  const int t = threadIdx.x, threads = blockDim.x;
  auto last = [&](int64_t incl) {  // the workgroup's total of an inclusive scan
    __syncthreads();
    if (t == threads - 1) lds.last = incl;
    __syncthreads();
    return lds.last;
  };
  // numbers up to `most`: their sum over the workgroup fits 32 bits, or takes two scans
  auto scan = [&](int v, int64_t most) -> int64_t {
    return most * threads <= INT32_MAX ? block_inclusive_scan(v, lds.scan) : block_inclusive_scan_wide(v, lds.scan);
  };
  int tiles = 0;
  for (int b0 = 0; b0 < p.B; b0 += threads) {
    int n = 0;
    if (b0 + t < p.B) {
      const Seq s = load_seq(p, b0 + t);
      const int64_t rows = (int64_t)s.n * p.g;
      n = rows > plan.min_rows ? (int)min<int64_t>((rows + plan.tile_rows - 1) / plan.tile_rows, plan.max_tiles) : 0;
    }
    const int64_t incl = tiles + scan(n, plan.max_tiles);
    const int end = (int)min<int64_t>(incl, plan.max_tiles);
    if (b0 + t < 1024) lds.end[b0 + t] = end;
    if (b0 + t < p.B) plan.tile_end[b0 + t] = end;
    tiles = (int)last(end);
  }
  __threadfence_block();
  __syncthreads();
  auto end_of = [&](int b) { return b < 1024 ? lds.end[b] : plan.tile_end[b]; };
  int64_t total = 0;
  int most = 0;
  for (int i0 = 0; i0 < tiles; i0 += threads) {
    const int i = i0 + t;
    int units = 0;
    if (i < tiles) {
      int lo = 0, hi = p.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (end_of(mid) > i)
          hi = mid;
        else
          lo = mid + 1;
      }
      const int qt = end_of(lo) - 1 - i;
      units = tile_range(p, load_seq(p, lo), qt, plan.tile_rows).units;
      plan.tile[i] = make_int2(lo, qt);
    }
    const int64_t incl = total + scan(units, p.num_keys / kTileKeys + 2);
    most = max(most, units);
    if (i < tiles) plan.unit_end[i] = incl;
    total = last(incl);
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) most = max(most, __shfl_xor(most, off, 64));
  if ((t & 63) == 0) lds.scan[t >> 6] = most;
  __syncthreads();
  for (int i = 0; i < threads / 64; ++i) most = max(most, lds.scan[i]);
  const float places = (float)plan.places, units = (float)total;
  const int64_t workers = max<int64_t>(1, min<int64_t>(plan.workers, total / kChunkMinUnits));
  // a unit's time with n workgroups at work, against that with all places taken
  const float per_cu = (float)plan.per_cu;
  auto pace = [&](float n) {
    return per_cu == 1.0f ? 1.0f : fmaxf(kLonePace, fminf(1.0f, __builtin_ceilf(n * per_cu / places) / per_cu));
  };
  float whole = (float)most;  // units that a place takes in turn, expected
  if ((float)tiles > places) whole = fmaxf(whole, 1.8f * units / (float)tiles);
  const float runs = (float)workers, divided = units / runs * pace(runs) + kJoinUnits + kPartUnits * runs / places;
  const bool divide = workers > 1 && (float)tiles < kWholeTiles * places && divided < whole * pace((float)tiles);
  if (t == 0) {
    plan.info[0] = divide ? workers : tiles;
    plan.info[1] = divide;
    plan.info[2] = total;
  }
  if (!divide) return;
  __threadfence_block();
  __syncthreads();
  for (int64_t w = t; w < workers; w += threads) {
    const int64_t x = w * total / workers;
    int lo = 0, hi = tiles - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (plan.unit_end[mid] > x)
        hi = mid;
      else
        lo = mid + 1;
    }
    plan.run_tile[w] = lo;
  }
}

}  // namespace nvq
