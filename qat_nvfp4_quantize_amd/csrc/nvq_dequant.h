// Exact fp16 dequantization of NVFP4 codes in registers, for the MFMA kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvq {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));

// E4M3 code byte b (0..3) of a dword -> fp16x2 pattern (code << 7) in both
// halves, i.e. s_b * 2^-8 twice.
__device__ __forceinline__ uint32_t scale_pair(uint32_t four, int b) {
  const uint32_t sel = (uint32_t)b | (0x0Cu << 8) | ((uint32_t)b << 16) | (0x0Cu << 24);
  return __builtin_amdgcn_perm(0u, four, sel) << 7;
}

// 8 FP4 codes (one dword) times the fp16x2 scale pattern -> 8 exact fp16 values.
__device__ __forceinline__ half8_t dequant8(uint32_t w, uint32_t pat) {
  half2_t s;
  __builtin_memcpy(&s, &pat, 4);
  const half2_t h0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 0) * s;
  const half2_t h1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 1) * s;
  const half2_t h2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 2) * s;
  const half2_t h3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 3) * s;
  half8_t r;
  r[0] = h0[0]; r[1] = h0[1]; r[2] = h1[0]; r[3] = h1[1];
  r[4] = h2[0]; r[5] = h2[1]; r[6] = h3[0]; r[7] = h3[1];
  return r;
}

}  // namespace nvq
