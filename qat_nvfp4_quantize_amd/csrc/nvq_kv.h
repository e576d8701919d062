// The paged NVFP4 KV cache as the kernels see it, and its host-side checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvq.h"
#include "nvq_internal.h"

namespace nvq {

struct KvPages {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const float *k_st, *v_st;
  int64_t num_pages, num_slots;
  int ps, log_ps, H, D;
};

// Checks a caller's cache and fills `c`.  by_slot: slots are addressed by
// int32 numbers, so all of them have to fit.
inline int kv_pages(const nvq_kv_cache* in, bool by_slot, KvPages& c) {
  if (!in || in->struct_size != sizeof(nvq_kv_cache)) return NVQ_EINVAL;
  const int ps = in->page_size, D = in->head_dim;
  if (ps < 16 || ps > 65536 || (ps & (ps - 1)) || D < 16 || D > 512 || (D & 15) || in->heads < 1 ||
      in->heads > 65535 || in->num_pages < 1 || in->num_pages > INT32_MAX)
    return NVQ_ESHAPE;
  if (by_slot && in->num_pages > INT32_MAX / ps) return NVQ_ESHAPE;
  if (!in->k_codes || !in->k_scales || !in->v_codes || !in->v_scales || !in->k_tensor_scale || !in->v_tensor_scale)
    return NVQ_EINVAL;
  if (!aligned16(in->k_codes) || !aligned16(in->k_scales) || !aligned16(in->v_codes) || !aligned16(in->v_scales) ||
      (((uintptr_t)in->k_tensor_scale | (uintptr_t)in->v_tensor_scale) & 3u))
    return NVQ_EALIGN;
  c.k_codes = in->k_codes, c.k_scales = in->k_scales, c.v_codes = in->v_codes, c.v_scales = in->v_scales;
  c.k_st = in->k_tensor_scale, c.v_st = in->v_tensor_scale;
  c.num_pages = in->num_pages;
  c.num_slots = in->num_pages * ps;
  c.ps = ps, c.H = in->heads, c.D = D;
  c.log_ps = __builtin_ctz((unsigned)ps);
  return NVQ_OK;
}

}  // namespace nvq
