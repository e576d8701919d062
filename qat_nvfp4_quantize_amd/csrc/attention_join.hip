// Joins the parts that the attention kernels leave of sequences and row tiles
// divided between workgroups: part i holds the unnormalised sum o_i, the sum
// of weights l_i and their reference m_i (powers of two), and
//   out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i.
// Bound by the parts' bytes and the latency of finding them; one launch for
// both kernels.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "nvq.h"
#include "nvq_attn.h"
#include "nvq_device.h"
#include "nvq_internal.h"

namespace nvq {
namespace {

constexpr int kJoinRows = 4;    // rows of a workgroup's step in a divided tile
constexpr int kJoinGroups = 16;  // workgroups per cut and head

template <int D>
struct JoinLds {
  float o[4][kJoinRows][D];
  float m[4][kJoinRows], l[4][kJoinRows];
};

// The four waves of a workgroup join R rows: wave w takes parts w, w + 4, ..;
// row k of part i is row `at(i) + k` of the buffers.  `out_row(k)` gives the
// query row and head, or a negative row.
template <int D, int R, class At, class OutRow>
__device__ __forceinline__ void join_rows(const AttnParams& p, const float2* part_ml, const float* part_o, int count,
                                          JoinLds<D>& lds, At at, OutRow out_row) {
  constexpr int kE = D / 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  float m[R], l[R], o[R][kE];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    m[k] = -INFINITY, l[k] = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[k][e] = 0.0f;
  }
#pragma unroll (R == 1 ? 8 : 2)
  for (int i = wave; i < count; i += 4)
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float2 ml = part_ml[at(i) + k];
      const float top = fmaxf(m[k], ml.x), ref = top == -INFINITY ? 0.0f : top;
      const float keep = __builtin_amdgcn_exp2f(m[k] - ref), f = __builtin_amdgcn_exp2f(ml.x - ref);
      m[k] = top;
      l[k] = l[k] * keep + ml.y * f;
#pragma unroll
      for (int e = 0; e < kE; ++e) o[k][e] = o[k][e] * keep + part_o[(at(i) + k) * D + kE * lane + e] * f;
    }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (lane == 0) lds.m[wave][k] = m[k], lds.l[wave][k] = l[k];
#pragma unroll
    for (int e = 0; e < kE; ++e) lds.o[wave][k][kE * lane + e] = o[k][e];
  }
  __syncthreads();
  const int k = wave;  // a row per wave
  int64_t row = -1;
  int head = 0;
  if (k < R) out_row(k, row, head);
  if (row >= 0) {
    const float top = fmaxf(fmaxf(lds.m[0][k], lds.m[1][k]), fmaxf(lds.m[2][k], lds.m[3][k]));
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, x[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) x[e] = 0.0f;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float f = __builtin_amdgcn_exp2f(lds.m[v][k] - ref);
      sum += lds.l[v][k] * f;
#pragma unroll
      for (int e = 0; e < kE; ++e) x[e] += lds.o[v][k][kE * lane + e] * f;
    }
    const OutScale scale(sum, *p.c.v_st);
    uint16_t* out = p.out + row * p.out_ld_t + head * p.out_ld_h + kE * lane;
#pragma unroll
    for (int e = 0; e < kE; ++e) out[e] = (uint16_t)scale.bf16(x[e]);
    if (p.lse && lane == 0)
      p.lse[row * p.Hq + head] = sum == 0.0f ? -INFINITY : (top + __builtin_log2f(sum)) * kLn2;
  }
  __syncthreads();
}

// blockIdx.y: key/value head; blockIdx.x: first the rows of the few-rows
// sequences, then the many-rows cuts, kJoinGroups blocks each.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnParams p, RowsPlan rows, ChunkPlan chunk, int row_blocks,
                                                   int blocks_per_seq, int row_step) {
  __shared__ JoinLds<D> lds;
  const int kvh = blockIdx.y;
  if ((int)blockIdx.x < row_blocks) {
    const int b = blockIdx.x / blocks_per_seq, r0 = (int)(blockIdx.x % blocks_per_seq) * row_step;
    const Seq s = load_seq(p, b);
    const int64_t n = (int64_t)s.n * p.g;
    if (r0 >= n || n > rows.max_rows) return;
    const int first = rows.seq[2 * b], count = rows.seq[2 * b + 1];
    if (count == 1) return;
    // the first worker's slot as noted, slot 0 of the others
    auto at = [&](int i) {
      return ((int64_t)(i == 0 ? first : 2 * ((first >> 1) + i)) * p.c.H + kvh) * rows.part_rows + r0;
    };
    auto out_row = [&](int k, int64_t& row, int& head) {
      const int r = r0 + k;
      row = r < n ? s.row0 + r / p.g : -1;
      head = kvh * p.g + r % p.g;
    };
    if (row_step == 1)
      join_rows<D, 1>(p, rows.part_ml, rows.part_o, count, lds, at, out_row);
    else
      join_rows<D, kJoinRows>(p, rows.part_ml, rows.part_o, count, lds, at, out_row);
    return;
  }
  // The cut between runs w - 1 and w.  A tile's cuts share its rows out.
  const int block = blockIdx.x - row_blocks;
  const int64_t w = block / kJoinGroups + 1, runs = chunk.info[0], total = chunk.info[2];
  if (chunk.info[1] == 0 || w >= runs) return;
  const int tile = chunk.run_tile[w];
  const int64_t end = chunk.unit_end[tile], start = tile ? chunk.unit_end[tile - 1] : 0;
  if (w * total / runs == start) return;  // between two tiles
  // runs of its first and last unit
  const int64_t w0 = ((start + 1) * runs - 1) / total, w1 = (end * runs - 1) / total;
  const int64_t first = 2 * w0 + (w0 * total / runs != start);
  const int2 bq = chunk.tile[tile];
  const Seq s = load_seq(p, bq.x);
  const int64_t n = (int64_t)s.n * p.g;
  for (int64_t g = (w - 1 - w0) * kJoinGroups + block % kJoinGroups; g * kJoinRows < chunk.tile_rows;
       g += (w1 - w0) * kJoinGroups) {
    const int64_t r0 = (int64_t)bq.y * chunk.tile_rows + g * kJoinRows;
    if (r0 < 0 || r0 >= n) return;
    join_rows<D, kJoinRows>(
        p, chunk.part_ml, chunk.part_o, (int)(w1 - w0) + 1, lds,
        [&](int i) { return ((i == 0 ? first : 2 * (w0 + i)) * p.c.H + kvh) * chunk.tile_rows + g * kJoinRows; },
        [&](int k, int64_t& row, int& head) {
          const int64_t r = r0 + k;
          row = r < n ? s.row0 + r / p.g : -1;
          head = kvh * p.g + (int)(r % p.g);
        });
  }
}

}  // namespace

int attn_join_launch(const AttnParams& p, const RowsPlan* rows, const ChunkPlan* chunk, hipStream_t s) {
  int row_blocks = 0, per_seq = 1, cut_blocks = 0, step = kJoinRows;
  if (rows && rows->may_split) {
    // Rows of one long context are few and have a part from every worker: a
    // workgroup each, with more loads in flight (131072 keys: 43 us against 47
    // by fours).  Many rows of few parts go by fours (33 drafts: 26 against 30).
    const int64_t n = std::min<int64_t>((int64_t)p.max_q * p.g, rows->max_rows);
    const int64_t by_fours = (n + kJoinRows - 1) / kJoinRows;
    step = p.B * by_fours * p.c.H < device_cu_count() ? 1 : kJoinRows;
    per_seq = (int)(step == 1 ? n : by_fours);
    row_blocks = p.B * per_seq;
  }
  if (chunk) cut_blocks = (chunk->workers - 1) * kJoinGroups;
  if (row_blocks + cut_blocks == 0) return NVQ_OK;
  const dim3 grid((unsigned)(row_blocks + cut_blocks), (unsigned)p.c.H);
  const RowsPlan r = rows ? *rows : RowsPlan{};
  const ChunkPlan c = chunk ? *chunk : ChunkPlan{};
  if (p.c.D == 64)
    hipLaunchKernelGGL(k_attn_join<64>, grid, dim3(256), 0, s, p, r, c, row_blocks, per_seq, step);
  else if (p.c.D == 128)
    hipLaunchKernelGGL(k_attn_join<128>, grid, dim3(256), 0, s, p, r, c, row_blocks, per_seq, step);
  else
    hipLaunchKernelGGL(k_attn_join<256>, grid, dim3(256), 0, s, p, r, c, row_blocks, per_seq, step);
  return last_launch();
}

}  // namespace nvq
