// Paged NVFP4 KV cache: new K and V tokens quantized as they are written into
// their slots, and slots read back.
//
// Both kernels are HBM-bound (2 or 4 bytes a value against 0.5625).  A
// workgroup takes consecutive tokens of one head, and workgroups are numbered heads first: they go to the eight XCDs in
// turn, so with 8 heads (or 4) an XCD sees one head (or half of its tokens).
// A token's V scales are single bytes in lines that the head's other slots
// share; kept to one L2 they are merged there.  32768 tokens of 8 heads x 128
// bf16 (172 MB at the least): 36 us with whole pages in order (4.8 TB/s), 54
// with slots in random order, against 45 and 62 with workgroups numbered
// tokens first.
//
// This translation unit is compiled with -ffp-contract=off (nvq_quant_block.h).

#include <hip/hip_runtime.h>

#include <algorithm>

#include "nvq.h"
#include "nvq_device.h"
#include "nvq_internal.h"
#include "nvq_kv.h"
#include "nvq_quant_block.h"

namespace nvq {
namespace {

constexpr int kKvThreads = 256;

// Token groups over y and z (y alone stops at 65535).
constexpr int kGroupsY = 32768;
__device__ __forceinline__ int64_t token_group() { return (int64_t)blockIdx.z * gridDim.y + blockIdx.y; }
dim3 kv_grid(const KvPages& c, int64_t T, int rows, int parts) {
  const int64_t groups = (T + rows - 1) / rows, y = std::min<int64_t>(groups, kGroupsY);
  return dim3((unsigned)(parts * c.H), (unsigned)y, (unsigned)((groups + y - 1) / y));
}

struct KvAppendParams {
  KvPages c;
  const char* src[2];        // k, v
  int64_t ld_t[2], ld_h[2];  // bytes
  const int32_t* slots;
  int64_t T;
  int rows;  // tokens of a workgroup's step: kKvThreads / (D / 16)
  uint32_t* status;
};

// Grid: x = head (K) or H + head (V), y and z the token group.  One block a
// thread (4 tokens a thread, loaded ahead, measured 59 us against 54).
template <bool kBF16>
__global__ __launch_bounds__(kKvThreads) void k_kv_append(KvAppendParams p) {
  __shared__ uint32_t s_slot[kKvThreads * (kBF16 ? 8 : 16)];
  const int nb = p.c.D >> 4;
  const bool is_v = (int)blockIdx.x >= p.c.H;
  const int h = blockIdx.x - (is_v ? p.c.H : 0);
  const int r = threadIdx.x / nb, blk = threadIdx.x - r * nb;
  const int64_t t = token_group() * p.rows + r;
  uint32_t bad = 0;
  if (r < p.rows && t < p.T) {
    const int32_t slot = p.slots[t];
    if (slot >= 0 && slot < p.c.num_slots) {
      RowBlock<kBF16> rb;
      rb.load_at(p.src[is_v] + t * p.ld_t[is_v] + h * p.ld_h[is_v] + blk * (kBF16 ? 32 : 64));
      const float s_t = *(is_v ? p.c.v_st : p.c.k_st);
      const double six_st = 6.0 * (double)s_t;
      const bool fast = (s_t >= 0x1p-100f) && (s_t <= 0x1p100f);
      uint32_t* lds = s_slot + threadIdx.x * (kBF16 ? 8 : 16);
      float acc[16];  // no residual sums on this path
      uint32_t sc, nonfinite = 0;
      uint2 cw;
      if (fast)
        encode_block_fast<kBF16, false>(rb, s_t, (float)(1.0 / six_st), (float)(1.0 / (double)s_t), sc, cw, acc,
                                        nonfinite, lds);
      else
        encode_block_exact<kBF16, false>(rb, s_t, six_st, sc, cw, acc, nonfinite, lds);
      if (nonfinite) bad |= (uint32_t)NVQ_STATUS_NONFINITE;
      const int off = slot & (p.c.ps - 1);
      const int64_t tile = ((int64_t)(slot >> p.c.log_ps) * p.c.H + h) << p.c.log_ps;  // first row of (page, head)
      *reinterpret_cast<uint2*>((is_v ? p.c.v_codes : p.c.k_codes) + ((tile + off) * nb + blk) * 8) = cw;
      if (is_v)
        p.c.v_scales[tile * nb + ((int64_t)blk << p.c.log_ps) + off] = (uint8_t)sc;
      else
        p.c.k_scales[(tile + off) * nb + blk] = (uint8_t)sc;
    } else if (slot >= 0) {
      bad |= (uint32_t)NVQ_STATUS_BAD_SLOT;
    }
  }
  bad = wave_or_u32(bad);
  if (bad && p.status && (threadIdx.x & 63) == 0) atomicOr(p.status, bad);
}

struct KvGatherParams {
  KvPages c;
  char* dst[2];  // k_out, v_out; NULL: not wanted
  const int32_t* slots;
  int64_t T;
  int rows;  // tokens of a workgroup's step
  int z0;  // first of the wanted outputs
  uint32_t* status;
};

// A thread writes 16 bytes (8 bf16 or 4 fp32 values) of kTok tokens, so a
// wave's stores are whole lines.
template <bool kBF16, int kTok>
__global__ __launch_bounds__(kKvThreads) void k_kv_gather(KvGatherParams p) {
  constexpr int kN = kBF16 ? 8 : 4;
  const int vecs = p.c.D / kN, nb = p.c.D >> 4;
  const bool second = (int)blockIdx.x >= p.c.H, is_v = second || p.z0;
  const int h = blockIdx.x - (second ? p.c.H : 0);
  const int r = threadIdx.x / vecs, vec = threadIdx.x - r * vecs, blk = vec * kN / 16;
  const int64_t t0 = token_group() * (kTok * p.rows) + r;
  uint32_t bad = 0;
  if (r < p.rows) {
    int32_t slot[kTok];
    uint32_t w[kTok], sc[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const int64_t t = t0 + i * p.rows;
      slot[i] = t < p.T ? p.slots[t] : -1;
    }
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      w[i] = sc[i] = 0u;
      if (slot[i] >= 0 && slot[i] < p.c.num_slots) {
        const int off = slot[i] & (p.c.ps - 1);
        const int64_t tile = ((int64_t)(slot[i] >> p.c.log_ps) * p.c.H + h) << p.c.log_ps;
        const uint8_t* at = (is_v ? p.c.v_codes : p.c.k_codes) + (tile + off) * (p.c.D >> 1) + vec * (kN / 2);
        w[i] = kBF16 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
        sc[i] = is_v ? p.c.v_scales[tile * nb + ((int64_t)blk << p.c.log_ps) + off]
                     : p.c.k_scales[(tile + off) * nb + blk];
      } else if (slot[i] >= 0) {
        bad = (uint32_t)NVQ_STATUS_BAD_SLOT;
      }
    }
    const float s_t = *(is_v ? p.c.v_st : p.c.k_st);
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const int64_t t = t0 + i * p.rows;
      if (t >= p.T) break;
      const float s_b = e4m3_to_f32(sc[i]);
      const float2 a = fp4_pair_to_f32<0>(w[i]), b = fp4_pair_to_f32<1>(w[i]);
      uint4 out;
      if constexpr (kBF16) {
        const float2 c = fp4_pair_to_f32<2>(w[i]), d = fp4_pair_to_f32<3>(w[i]);
        auto two = [&](float2 g) {
          return f32_to_bf16_rne((g.x * s_b) * s_t) | (f32_to_bf16_rne((g.y * s_b) * s_t) << 16);
        };
        out = make_uint4(two(a), two(b), two(c), two(d));
      } else {
        auto one = [&](float g) { return __float_as_uint((g * s_b) * s_t); };
        out = make_uint4(one(a.x), one(a.y), one(b.x), one(b.y));
      }
      *reinterpret_cast<uint4*>(p.dst[is_v] + (((t * p.c.H + h) * vecs) + vec) * 16) = out;
    }
  }
  bad = wave_or_u32(bad);
  if (bad && p.status && (threadIdx.x & 63) == 0) atomicOr(p.status, bad);
}

// Four tokens a thread where that leaves every CU a few workgroups (32768
// tokens in page order: 41 us against 49 with one; in random order 56 and 62,
// most of it lines read for 64 of their 128 bytes and for single V scales).
constexpr int kManyTokens = 4;
bool many_tokens(const KvPages& c, int64_t T, int rows) {
  return 2 * c.H * (T / (kManyTokens * rows)) >= 4 * (int64_t)device_cu_count();
}

int check_ws(void* ws, size_t ws_bytes) {
  if (!ws) return NVQ_OK;
  if (!aligned256(ws)) return NVQ_EALIGN;
  return ws_bytes < kAlign ? NVQ_EWORKSPACE : NVQ_OK;
}

}  // namespace
}  // namespace nvq

using namespace nvq;

extern "C" int nvq_kv_append(const nvq_kv_cache* cache, const void* k, const void* v, int dtype, int64_t T,
                             int64_t k_ld_t, int64_t k_ld_h, int64_t v_ld_t, int64_t v_ld_h,
                             const int32_t* slots, void* ws, size_t ws_bytes, void* stream) {
  KvAppendParams p{};
  if (int rc = kv_pages(cache, true, p.c)) return rc;
  if (dtype != NVQ_F32 && dtype != NVQ_BF16) return NVQ_EINVAL;
  if (T < 0 || T > kMaxTokens) return NVQ_ESHAPE;
  const int64_t es = dtype == NVQ_BF16 ? 2 : 4;
  const int64_t ld[4] = {k_ld_t ? k_ld_t : (int64_t)p.c.H * p.c.D, k_ld_h ? k_ld_h : p.c.D,
                         v_ld_t ? v_ld_t : (int64_t)p.c.H * p.c.D, v_ld_h ? v_ld_h : p.c.D};
  for (int64_t l : ld) {
    if (l < 0) return NVQ_ESHAPE;
    if (l * es % 16) return NVQ_EALIGN;
  }
  if (int rc = check_ws(ws, ws_bytes)) return rc;
  if (T > 0 && (!k || !v || !slots)) return NVQ_EINVAL;
  if (!aligned16(k) || !aligned16(v) || ((uintptr_t)slots & 3u)) return NVQ_EALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (ws)
    if (int rc = clear_status(static_cast<uint32_t*>(ws), s)) return rc;
  if (T == 0) return NVQ_OK;
  p.src[0] = static_cast<const char*>(k), p.src[1] = static_cast<const char*>(v);
  p.ld_t[0] = ld[0] * es, p.ld_h[0] = ld[1] * es, p.ld_t[1] = ld[2] * es, p.ld_h[1] = ld[3] * es;
  p.slots = slots, p.T = T;
  p.rows = kKvThreads / (p.c.D / 16);
  p.status = static_cast<uint32_t*>(ws);
  const dim3 grid = kv_grid(p.c, T, p.rows, 2);
  if (dtype == NVQ_BF16)
    hipLaunchKernelGGL(k_kv_append<true>, grid, dim3(kKvThreads), 0, s, p);
  else
    hipLaunchKernelGGL(k_kv_append<false>, grid, dim3(kKvThreads), 0, s, p);
  return last_launch();
}

extern "C" int nvq_kv_gather(const nvq_kv_cache* cache, const int32_t* slots, int64_t T, void* k_out, void* v_out,
                             int out_dtype, void* ws, size_t ws_bytes, void* stream) {
  KvGatherParams p{};
  if (int rc = kv_pages(cache, true, p.c)) return rc;
  if (out_dtype != NVQ_F32 && out_dtype != NVQ_BF16) return NVQ_EINVAL;
  if (T < 0 || T > kMaxTokens) return NVQ_ESHAPE;
  if (int rc = check_ws(ws, ws_bytes)) return rc;
  if (T > 0 && (!slots || (!k_out && !v_out))) return NVQ_EINVAL;
  if (!aligned16(k_out) || !aligned16(v_out) || ((uintptr_t)slots & 3u)) return NVQ_EALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (ws)
    if (int rc = clear_status(static_cast<uint32_t*>(ws), s)) return rc;
  if (T == 0) return NVQ_OK;
  p.dst[0] = static_cast<char*>(k_out), p.dst[1] = static_cast<char*>(v_out);
  p.slots = slots, p.T = T;
  const bool bf16 = out_dtype == NVQ_BF16;
  p.rows = kKvThreads / (p.c.D / (bf16 ? 8 : 4));
  p.z0 = k_out ? 0 : 1;
  p.status = static_cast<uint32_t*>(ws);
  const bool many = many_tokens(p.c, T, p.rows);
  const dim3 grid = kv_grid(p.c, T, p.rows * (many ? kManyTokens : 1), k_out && v_out ? 2 : 1);
  if (bf16 && many)
    hipLaunchKernelGGL((k_kv_gather<true, kManyTokens>), grid, dim3(kKvThreads), 0, s, p);
  else if (bf16)
    hipLaunchKernelGGL((k_kv_gather<true, 1>), grid, dim3(kKvThreads), 0, s, p);
  else if (many)
    hipLaunchKernelGGL((k_kv_gather<false, kManyTokens>), grid, dim3(kKvThreads), 0, s, p);
  else
    hipLaunchKernelGGL((k_kv_gather<false, 1>), grid, dim3(kKvThreads), 0, s, p);
  return last_launch();
}
