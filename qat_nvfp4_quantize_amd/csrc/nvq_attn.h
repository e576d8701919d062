// What the attention kernels share: the call's parameters, the sequences as
// the device sees them and the check of the index arrays.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvq.h"
#include "nvq_device.h"
#include "nvq_kv.h"
#include "nvq_scan.h"

namespace nvq {

struct AttnParams {
  KvPages c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const int32_t *cu_q, *kv_len, *table;
  int64_t q_ld_t, q_ld_h, out_ld_t, out_ld_h, table_ld;
  int64_t window;    // 0: none
  int64_t num_keys;  // keys a row of the block table covers
  int total_q, B, max_q, Hq, g;
  int causal;
  float scale_log2;  // softmax_scale * log2(e)
  uint32_t* status;
};

// Plan of the few-rows kernel, and where the parts of split sequences go.
struct RowsPlan {
  int max_rows;  // sequences with more rows per key/value head are left out
  int workers;   // most of them per key/value head
  int waves;     // of a worker: 4, or 1 (four workers a workgroup)
  int whole;     // a worker is a sequence
  int may_split;
  int part_rows;  // rows of a part
  int plans_chunks;  // the launch has a workgroup that plans the many-rows one
  int32_t* seq;     // [B][2]: first worker and its slot (2 worker + slot), number of workers
  float2* part_ml;  // [worker][2 slots][head][part_rows] reference and sum
  float* part_o;    // [worker][2 slots][head][part_rows][D]
};

int attn_rows_tiles(int D, int64_t rows);
void attn_rows_plan(const AttnParams& p, int tiles, bool chunks, WsCarve& ws, RowsPlan& plan);

// Plan of the many-rows kernel: row tiles and their key tiles in one
// row of units per key/value head, cut into runs, and where the parts of tiles
// that a cut divides go.
struct ChunkPlan {
  int min_rows;  // sequences with no more rows per key/value head are left out
  int check;     // the launch checks the index arrays
  int places;    // workgroups that the chip holds, per key/value head
  int per_cu;    // and per CU
  int workers;   // most runs per key/value head where tiles are divided
  int tile_rows;  // 128 or 256
  int64_t max_tiles;
  int32_t* tile_end;   // [B] row tiles up to and with sequence b
  int2* tile;          // [max_tiles] sequence, row tile in it
  int64_t* unit_end;   // [max_tiles] units up to and with a tile
  int32_t* run_tile;   // [workers] tile of a run's first unit
  int64_t* info;       // runs, whether tiles are divided, units in all
  float2* part_ml;     // [run][2 slots][head][tile_rows] reference and sum
  float* part_o;       // [run][2 slots][head][tile_rows][D]
};

void attn_chunk_plan(const AttnParams& p, int min_rows, bool check, WsCarve& ws, ChunkPlan& plan);
int attn_chunk_launch(const AttnParams& p, const ChunkPlan& plan, bool planned, hipStream_t s);
int attn_rows_launch(const AttnParams& p, const RowsPlan& plan, const ChunkPlan& chunk, hipStream_t s);
// Joins what either kernel left in parts (a NULL plan: that kernel did not run).
int attn_join_launch(const AttnParams& p, const RowsPlan* rows, const ChunkPlan* chunk, hipStream_t s);

constexpr float kLn2 = 0.69314718055994530942f;

// An output is a sum of weighted codes divided by the sum of weights, times V's
// tensor scale.  In two factors: sums of weights pass 2^26, and a small scale
// divided by that is no normal number though the output is one.  No weight at
// all (no key seen): zeros, whatever the scale.
struct OutScale {
  float inv, st;
  __device__ __forceinline__ OutScale(float sum, float v_st)
      : inv(sum == 0.0f ? 0.0f : 1.0f / sum), st(sum == 0.0f ? 0.0f : v_st) {}
  __device__ __forceinline__ uint32_t bf16(float x) const { return f32_to_bf16_any(x * inv * st); }
};

// Rows and keys of sequence b, cut to what the call's buffers hold.
struct Seq {
  int row0, n;   // query rows
  int64_t len;   // keys
  int64_t pos0;  // position of the first row: the rows are the last positions
};
__device__ __forceinline__ Seq load_seq(const AttnParams& p, int b) {
  Seq s;
  s.row0 = min(max(p.cu_q[b], 0), p.total_q);
  const int n = max(min(p.cu_q[b + 1], p.total_q) - s.row0, 0);
  s.n = min(n, p.max_q);
  s.len = max(p.kv_len[b], 0);
  s.pos0 = s.len - n;
  return s;
}

// Visible keys [lo, hi) of the query at position pos.
__device__ __forceinline__ void visible(const AttnParams& p, const Seq& s, int64_t pos, int64_t& lo, int64_t& hi) {
  hi = min(p.causal ? pos + 1 : s.len, min(s.len, p.num_keys));
  lo = p.window > 0 ? max<int64_t>(pos - p.window + 1, 0) : 0;
}

// One workgroup looks over the index arrays and writes the status word:
// lengths and row ranges of every sequence, and the page id of every page
// that some query row of it can see.  It runs beside the others, which only
// stay inside the buffers, so no atomic and no clearing is needed.  A batch
// of 256 sequences at a time, a thread each, then the pages of all of them in
// one run, so that few loads wait for one another (64 sequences of 64 pages:
// 17 us with a loop over the sequences, hidden now).  All kThreads threads of
// the workgroup call it: those past the batch add nothing to the scan.
constexpr int kCheckBatch = 256;
struct CheckLds {
  int end[kCheckBatch];  // pages of the batch's sequences up to and with this one
  int first[kCheckBatch];
  int wave[16];
  uint32_t flag;
};
template <int kThreads>
__device__ __forceinline__ void check_batch(const AttnParams& p, CheckLds& lds) {
  static_assert(kThreads >= kCheckBatch);
  const int t = threadIdx.x;
  const bool in_batch = kThreads == kCheckBatch || t < kCheckBatch;
  if (t == 0) lds.flag = 0u;
  bool bad = false;
  for (int b0 = 0; b0 < p.B; b0 += kCheckBatch) {
    const int b = b0 + t;
    int first = 0, n = 0;
    if (in_batch && b < p.B) {
      const int64_t r0 = p.cu_q[b], r1 = p.cu_q[b + 1], len = p.kv_len[b];
      bad |= r0 < 0 || r1 < r0 || r1 > p.total_q || r1 - r0 > p.max_q || len < 0 || (r1 > r0 && len > p.num_keys);
      const Seq s = load_seq(p, b);
      if (s.n > 0) {
        int64_t lo, hi, x;
        visible(p, s, s.pos0, lo, x);
        visible(p, s, s.pos0 + s.n - 1, x, hi);
        if (hi > lo) {
          first = (int)(lo >> p.c.log_ps);
          n = (int)((hi - 1) >> p.c.log_ps) + 1 - first;
        }
      }
    }
    __syncthreads();
    if (in_batch) lds.first[t] = first;
    const int incl = block_inclusive_scan(n, lds.wave);
    if (in_batch) lds.end[t] = incl;
    __syncthreads();
    const int all = lds.end[kCheckBatch - 1];
#pragma unroll 4
    for (int i = t; i < all; i += kThreads) {
      int lo = 0, hi = kCheckBatch - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (lds.end[mid] > i)
          hi = mid;
        else
          lo = mid + 1;
      }
      const int at = lds.first[lo] + i - (lo ? lds.end[lo - 1] : 0);
      const int32_t id = p.table[(b0 + lo) * p.table_ld + at];
      bad |= id < 0 || id >= p.c.num_pages;
    }
  }
  __syncthreads();
  if (bad) atomicOr(&lds.flag, (uint32_t)NVQ_STATUS_BAD_SEQUENCE);
  __syncthreads();
  if (t == 0) *p.status = lds.flag;
}

}  // namespace nvq
