// Attention of new tokens over the paged NVFP4 KV cache.
//
// Mathematics: for a query row q at position p and its visible keys j,
//   out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = c q . k_j,
// c = softmax_scale log2(e) s_tK, over one pass of the keys with a running
// reference m and sum; parts of the keys are joined by rescaling each to the
// common maximum.  A stored value is G s_b s_t: G s_b has at most 6
// significant bits, so it is exact in fp16, and s_t leaves the sums.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "nvq.h"
#include "nvq_attn.h"
#include "nvq_dequant.h"
#include "nvq_device.h"
#include "nvq_internal.h"
#include "nvq_kv.h"

namespace nvq {
namespace {

// ----------------------------------------------------------- any head size --
// One workgroup per query row and head, its four waves taking 64 keys each in
// turn.  Scores: a lane per key, the dot product in fp32 over the key's
// blocks.  Values: a lane per 64th element, over the wave's visible keys.
constexpr int kAnyMaxD = 512;

__global__ __launch_bounds__(256) void k_attn_any(AttnParams p) {
  __shared__ float s_q[kAnyMaxD];
  __shared__ float s_o[4][kAnyMaxD];
  __shared__ float s_ml[4][2];
  __shared__ CheckLds s_check;
  if (blockIdx.y == 0) {
    if (blockIdx.x == 0) check_batch<256>(p, s_check);
    return;
  }
  const int row = blockIdx.x, h = blockIdx.y - 1, kvh = h / p.g;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int D = p.c.D, nb = D >> 4;
  // the last sequence that starts at or before the row
  int lo_b = 0, hi_b = p.B;
  while (lo_b < hi_b) {
    const int mid = (lo_b + hi_b) >> 1;
    if (p.cu_q[mid + 1] <= row)
      lo_b = mid + 1;
    else
      hi_b = mid;
  }
  const int b = lo_b;
  if (b >= p.B) return;
  const Seq s = load_seq(p, b);
  if (row < s.row0 || row >= s.row0 + s.n) return;
  int64_t lo, hi;
  visible(p, s, s.pos0 + (row - s.row0), lo, hi);
  // Q under a power of two that brings its largest magnitude to 2^14 .. 2^15, as
  // in the other kernels: its products with stored values stay within fp32.
  // Every wave looks over the row itself.
  const uint16_t* q = p.q + row * p.q_ld_t + h * p.q_ld_h;
  uint32_t big = 0;
  for (int d = lane; d < D; d += 64) big = max(big, (uint32_t)q[d] & 0x7FFFu);
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) big = max(big, (uint32_t)__shfl_xor((int)big, x, 64));
  const int ex = (int)(big >> 7);
  const int shift = (big == 0u || ex == 255) ? 0 : 14 + 127 - max(ex, 1);
  for (int d = threadIdx.x; d < D; d += 256) s_q[d] = __builtin_ldexpf(bf16_to_f32(q[d]), shift);
  __syncthreads();
  const int32_t* table = p.table + b * p.table_ld;
  const float c = __builtin_ldexpf(p.scale_log2 * *p.c.k_st, -shift);
  float m = -INFINITY, l = 0.0f, o[kAnyMaxD / 64];
#pragma unroll
  for (int i = 0; i < kAnyMaxD / 64; ++i) o[i] = 0.0f;
  for (int64_t kb = lo + 64 * wave; kb < hi; kb += 256) {
    const int64_t j = kb + lane;
    const int32_t id = j < hi ? table[j >> p.c.log_ps] : -1;
    const bool see = id >= 0 && id < p.c.num_pages;
    const int64_t tile = see ? ((int64_t)id * p.c.H + kvh) << p.c.log_ps : 0;
    const int off = (int)(j & (p.c.ps - 1));
    float dot = 0.0f;
    if (see) {
      for (int blk = 0; blk < nb; ++blk) {
        const uint2 cw = *reinterpret_cast<const uint2*>(p.c.k_codes + ((tile + off) * nb + blk) * 8);
        const uint32_t s_b = scale_pair(p.c.k_scales[(tile + off) * nb + blk], 0);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const half8_t v = dequant8(i < 8 ? cw.x : cw.y, s_b);
          dot = fmaf((float)v[i & 7], s_q[blk * 16 + i], dot);
        }
      }
    }
    const float sc = see ? dot * c : -INFINITY;
    float top = sc;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x, 64));
    uint64_t seen = __ballot(see);
    if (!seen) continue;
    const float m_new = fmaxf(m, top);
    const float ref = m_new == -INFINITY ? 0.0f : m_new;
    const float keep = __builtin_amdgcn_exp2f(m - ref);  // 0 for m = -inf
    const float pj = see ? __builtin_amdgcn_exp2f(sc - ref) : 0.0f;
    m = m_new;
    float sum = pj;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x, 64);
    l = l * keep + sum;
#pragma unroll
    for (int i = 0; i < kAnyMaxD / 64; ++i) o[i] *= keep;
    while (seen) {
      const int k = __builtin_ctzll(seen);
      seen &= seen - 1;
      const float w = __shfl(pj, k, 64);
      const int64_t tk = __shfl(tile, k, 64);
      const int ok = __shfl(off, k, 64);
#pragma unroll
      for (int i = 0; i < kAnyMaxD / 64; ++i) {
        const int d = lane + 64 * i;
        if (d < D) {
          const uint32_t byte = p.c.v_codes[(tk + ok) * (int64_t)(D >> 1) + (d >> 1)];
          const uint32_t nib = (d & 1) ? byte >> 4 : byte & 15u;
          const float s_b = e4m3_to_f32(p.c.v_scales[tk * nb + ((int64_t)(d >> 4) << p.c.log_ps) + ok]);
          const float v = e2m1_mag(nib & 7u) * s_b;
          o[i] = fmaf(w, (nib & 8u) ? -v : v, o[i]);
        }
      }
    }
  }
  if (lane == 0) s_ml[wave][0] = m, s_ml[wave][1] = l;
#pragma unroll
  for (int i = 0; i < kAnyMaxD / 64; ++i)
    if (lane + 64 * i < D) s_o[wave][lane + 64 * i] = o[i];
  __syncthreads();
  float mx = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) mx = fmaxf(mx, s_ml[w][0]);
  const float ref = mx == -INFINITY ? 0.0f : mx;
  float f[4], sum = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = __builtin_amdgcn_exp2f(s_ml[w][0] - ref);
    sum += s_ml[w][1] * f[w];
  }
  const OutScale scale(sum, *p.c.v_st);
  uint16_t* out = p.out + row * p.out_ld_t + h * p.out_ld_h;
  for (int d = threadIdx.x; d < D; d += 256) {
    const float v = s_o[0][d] * f[0] + s_o[1][d] * f[1] + s_o[2][d] * f[2] + s_o[3][d] * f[3];
    out[d] = (uint16_t)scale.bf16(v);
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[(int64_t)row * p.Hq + h] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

constexpr float kLog2e = 1.44269504088896340736f;

// Host-side checks of the sizes (no HIP call, no pointer of args but sizes).
int attn_sizes(const nvq_kv_cache* cache, const nvq_paged_attention_args* a, AttnParams& p) {
  if (!cache || cache->struct_size != sizeof(nvq_kv_cache)) return NVQ_EINVAL;
  if (!a || a->struct_size != sizeof(nvq_paged_attention_args)) return NVQ_EINVAL;
  if (a->total_q < 0 || a->total_q > kMaxTokens || a->B < 0 || a->B > 65535 || a->max_q < 0 || a->table_width < 0)
    return NVQ_ESHAPE;
  const int ps = cache->page_size;
  if (cache->heads < 1 || ps < 16 || ps > 65536 || a->q_heads < 1 || a->q_heads > 32768 ||
      a->q_heads % cache->heads)
    return NVQ_ESHAPE;
  // counted in 32 bits: the keys of a sequence, the pages and 128-key units of
  // all, the threads of a launch
  if (a->table_width > INT32_MAX / ps || a->B * a->table_width > (1 << 30) ||
      a->B * (a->table_width * ps / 128 + 2) > INT32_MAX || a->B * cache->heads > (1 << 21) ||
      a->total_q * a->q_heads > (1 << 30))
    return NVQ_ESHAPE;
  p.total_q = (int)a->total_q, p.B = (int)a->B;
  p.max_q = (int)(a->max_q == 0 ? a->total_q : std::min(a->max_q, a->total_q));
  p.Hq = a->q_heads, p.g = a->q_heads / cache->heads;
  p.num_keys = a->table_width * ps;
  p.window = std::min<int64_t>(a->window, INT32_MAX);  // past every key; sums with it stay in range
  p.c.H = cache->heads, p.c.D = cache->head_dim;
  return NVQ_OK;
}

// Which kernels a call takes, and their workspace.  Head dimensions 64, 128
// and 256 go to the MFMA kernels: sequences of few rows per key/value head to
// the one that reads the pages into operands, the others to the one that
// shares dequantized tiles; a batch that may hold both kinds launches both,
// and each leaves the other's sequences out.  Other dimensions take one
// workgroup per row.
struct Plan {
  RowsPlan rows;
  ChunkPlan chunk;
  bool use_rows, use_chunk;
  size_t bytes;
};

Plan attn_plan(const AttnParams& p, void* ws) {
  Plan plan{};
  WsCarve c(ws);
  if (p.c.D == 64 || p.c.D == 128 || p.c.D == 256) {
    int tiles = attn_rows_tiles(p.c.D, (int64_t)p.max_q * p.g);
    plan.use_chunk = tiles == 0;
    if (plan.use_chunk && p.B > 1) tiles = attn_rows_tiles(p.c.D, p.g);  // single tokens beside the chunks
    plan.use_rows = tiles > 0;
    if (plan.use_rows) attn_rows_plan(p, tiles, plan.use_chunk, c, plan.rows);
    if (plan.use_chunk) attn_chunk_plan(p, 16 * tiles, !plan.use_rows, c, plan.chunk);
  }
  plan.bytes = c.off;
  return plan;
}

}  // namespace
}  // namespace nvq

using namespace nvq;

extern "C" size_t nvq_paged_attention_workspace_bytes(const nvq_kv_cache* cache,
                                                      const nvq_paged_attention_args* args) {
  AttnParams p{};
  if (attn_sizes(cache, args, p)) return kAlign;
  return attn_plan(p, nullptr).bytes;
}

extern "C" int nvq_paged_attention(const nvq_kv_cache* cache, const nvq_paged_attention_args* args, void* stream) {
  AttnParams p{};
  if (int rc = attn_sizes(cache, args, p)) return rc;
  if (int rc = kv_pages(cache, false, p.c)) return rc;
  const nvq_paged_attention_args& a = *args;
  const int D = p.c.D;
  if ((a.causal != 0 && a.causal != 1) || a.window < 0 || (a.window > 0 && !a.causal) ||
      !std::isfinite(a.softmax_scale * kLog2e))
    return NVQ_EINVAL;
  p.q_ld_t = a.q_ld_t ? a.q_ld_t : (int64_t)p.Hq * D;
  p.q_ld_h = a.q_ld_h ? a.q_ld_h : D;
  p.out_ld_t = a.out_ld_t ? a.out_ld_t : (int64_t)p.Hq * D;
  p.out_ld_h = a.out_ld_h ? a.out_ld_h : D;
  p.table_ld = a.table_ld ? a.table_ld : a.table_width;
  if (p.q_ld_t < 0 || p.q_ld_h < 0 || p.out_ld_t < 0 || p.out_ld_h < 0 || p.table_ld < a.table_width)
    return NVQ_ESHAPE;
  // rows of out must not overlap
  if ((p.Hq > 1 && p.out_ld_h < D) || (p.total_q > 1 && p.out_ld_t < D)) return NVQ_ESHAPE;
  if (p.Hq > 1 && p.total_q > 1 && p.out_ld_t < (p.Hq - 1) * p.out_ld_h + D &&
      p.out_ld_h < (p.total_q - 1) * p.out_ld_t + D)
    return NVQ_ESHAPE;
  if (p.q_ld_t % 8 || p.q_ld_h % 8 || p.out_ld_t % 8 || p.out_ld_h % 8 || !aligned16(a.q) || !aligned16(a.out) ||
      (((uintptr_t)a.cu_q | (uintptr_t)a.kv_len | (uintptr_t)a.block_table | (uintptr_t)a.lse) & 3u))
    return NVQ_EALIGN;
  if (!a.ws) return NVQ_EINVAL;
  if (!aligned256(a.ws)) return NVQ_EALIGN;
  const Plan plan = attn_plan(p, a.ws);
  if (a.ws_bytes < plan.bytes) return NVQ_EWORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  p.status = static_cast<uint32_t*>(a.ws);
  if (p.total_q == 0 || p.B == 0) return clear_status(p.status, s);
  if (!a.q || !a.out || !a.cu_q || !a.kv_len || (!a.block_table && a.table_width > 0)) return NVQ_EINVAL;
  p.q = a.q, p.out = a.out, p.lse = a.lse;
  p.cu_q = a.cu_q, p.kv_len = a.kv_len, p.table = a.block_table;
  p.causal = a.causal;
  p.scale_log2 = a.softmax_scale * kLog2e;
  if (plan.use_rows || plan.use_chunk) {
    if (plan.use_rows)
      if (int rc = attn_rows_launch(p, plan.rows, plan.chunk, s)) return rc;
    if (plan.use_chunk)
      if (int rc = attn_chunk_launch(p, plan.chunk, plan.use_rows, s)) return rc;
    return attn_join_launch(p, plan.use_rows ? &plan.rows : nullptr, plan.use_chunk ? &plan.chunk : nullptr, s);
  }
  hipLaunchKernelGGL(k_attn_any, dim3((unsigned)p.total_q, (unsigned)p.Hq + 1), dim3(256), 0, s, p);
  return last_launch();
}
