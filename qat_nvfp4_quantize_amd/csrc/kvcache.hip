// Paged NVFP4 KV cache: new K and V tokens quantized as they are written into
// their slots, and slots read back.
//
// Both kernels are HBM-bound (2 or 4 bytes a value against 0.5625), one
// 16-element block per thread.  A workgroup takes consecutive tokens of one
// head: where a sequence's tokens fill a page in order, the page's 64-byte
// code rows and the V scales (slots innermost) of those tokens are written by
// one workgroup, so one L2 merges them into whole lines.
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

struct KvAppendParams {
  KvPages c;
  const char* src[2];        // k, v
  int64_t ld_t[2], ld_h[2];  // bytes
  const int32_t* slots;
  int64_t T;
  int rows;  // tokens of a workgroup: kKvThreads / (D / 16), at least 1
  uint32_t* status;
};

// blockIdx: x token group, y head, z 0 for K and 1 for V.
template <bool kBF16>
__global__ __launch_bounds__(kKvThreads) void k_kv_append(KvAppendParams p) {
  __shared__ uint32_t s_slot[kKvThreads * (kBF16 ? 8 : 16)];
  const int nb = p.c.D >> 4, h = blockIdx.y;
  const int r = threadIdx.x / nb, blk = threadIdx.x - r * nb;
  const int64_t t = (int64_t)blockIdx.x * p.rows + r;
  uint32_t bad = 0;
  if (r < p.rows && t < p.T) {
    const int32_t slot = p.slots[t];
    if (slot >= 0 && slot < p.c.num_slots) {
      const bool is_v = blockIdx.z != 0;
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
      const int64_t page = slot >> p.c.log_ps;
      const int off = slot & (p.c.ps - 1);
      const int64_t tile = (page * p.c.H + h) << p.c.log_ps;  // first slot row of (page, head)
      *reinterpret_cast<uint2*>((is_v ? p.c.v_codes : p.c.k_codes) + ((tile + off) * nb + blk) * 8) = cw;
      if (is_v)
        p.c.v_scales[tile * nb + ((int64_t)blk << p.c.log_ps) + off] = (uint8_t)sc;
      else
        p.c.k_scales[(tile + off) * nb + blk] = (uint8_t)sc;
      if (nonfinite) bad |= (uint32_t)NVQ_STATUS_NONFINITE;
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
  int rows;
  int z0;  // first of the wanted outputs
  uint32_t* status;
};

template <bool kBF16>
__global__ __launch_bounds__(kKvThreads) void k_kv_gather(KvGatherParams p) {
  const int nb = p.c.D >> 4, h = blockIdx.y;
  const int r = threadIdx.x / nb, blk = threadIdx.x - r * nb;
  const int64_t t = (int64_t)blockIdx.x * p.rows + r;
  uint32_t bad = 0;
  if (r < p.rows && t < p.T) {
    const bool is_v = p.z0 + (int)blockIdx.z != 0;
    const int32_t slot = p.slots[t];
    uint2 cw = make_uint2(0u, 0u);
    float s_b = 0.0f;
    if (slot >= 0 && slot < p.c.num_slots) {
      const int64_t page = slot >> p.c.log_ps;
      const int off = slot & (p.c.ps - 1);
      const int64_t tile = (page * p.c.H + h) << p.c.log_ps;
      cw = *reinterpret_cast<const uint2*>((is_v ? p.c.v_codes : p.c.k_codes) + ((tile + off) * nb + blk) * 8);
      s_b = e4m3_to_f32(is_v ? p.c.v_scales[tile * nb + ((int64_t)blk << p.c.log_ps) + off]
                             : p.c.k_scales[(tile + off) * nb + blk]);
    } else if (slot >= 0) {
      bad = (uint32_t)NVQ_STATUS_BAD_SLOT;
    }
    const float s_t = *(is_v ? p.c.v_st : p.c.k_st);
    float v[16];
    block_values(cw, s_b, s_t, v);
    char* out = p.dst[is_v] + ((t * p.c.H + h) * nb + blk) * (kBF16 ? 32 : 64);
    store_block<kBF16>(v, out);
  }
  bad = wave_or_u32(bad);
  if (bad && p.status && (threadIdx.x & 63) == 0) atomicOr(p.status, bad);
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
  const dim3 grid((unsigned)((T + p.rows - 1) / p.rows), (unsigned)p.c.H, 2);
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
  p.rows = kKvThreads / (p.c.D / 16);
  p.z0 = k_out ? 0 : 1;
  p.status = static_cast<uint32_t*>(ws);
  const dim3 grid((unsigned)((T + p.rows - 1) / p.rows), (unsigned)p.c.H, (k_out && v_out) ? 2 : 1);
  if (out_dtype == NVQ_BF16)
    hipLaunchKernelGGL(k_kv_gather<true>, grid, dim3(kKvThreads), 0, s, p);
  else
    hipLaunchKernelGGL(k_kv_gather<false>, grid, dim3(kKvThreads), 0, s, p);
  return last_launch();
}
