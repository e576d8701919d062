/*
 * nvq.h -- C ABI of libnvq.so: NVFP4 quantization, residual-channel selection,
 * W4A4 MoE grouped GEMM with residual compensation and asymmetric W4A16 QAT
 * GEMMs on AMD Instinct MI355X (gfx950).
 *
 * Method sources (cited by page and section; the pages print no equations):
 *  - QUADS explainer ("QUADS: Stabilizing NVFP4 Reinforcement Learning for MoE
 *    via QUantization-error Alignment across Dual Sides", gist.science):
 *      §1   NVFP4 W4A4 GEMMs, E2M1 grid with 8 magnitudes per sign;
 *      §2.1 weights take the same quantize-dequantize path on both sides,
 *           activations are quantized online;
 *      §2.2-A asymmetric W4A16 QAT: fake-quantized NVFP4 weights, BF16
 *           activations in the trainer forward;
 *      §2.2-B residual activation compensation: the channels with the largest
 *           quantization residual get a correction added to the W4A4 output.
 *  - TRACE post ("TRACE : un entraînement conscient de la quantification guidé
 *    par le rollout ...", sns.style), "Fonctionnement, côté ingénierie" and
 *    "L'idée centrale de TRACE": block-scaled FP4, the trainer takes its
 *    rounding from the rollout's recorded quantization (codes and scales).
 *  - NVFP4 layout the pages leave open: 16-element blocks along K, one E4M3
 *    (OCP FP8 "FN") scale per block, one fp32 scale per tensor
 *    s_t = amax / (6 * 448), E2M1 elements (OCP MX v1.0), round to nearest,
 *    ties to even, two codes per byte with the even element in the low nibble.
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers, row-major, owned by the caller.
 *    The library allocates nothing; scratch memory is the caller's workspace
 *    `ws` of `ws_bytes` bytes (size it with the matching *_workspace_bytes
 *    query; 256-byte aligned).
 *  - `stream` is a hipStream_t (NULL = the null stream).  Calls only enqueue
 *    work on it; none synchronizes the host.  Calls that share a workspace
 *    must be ordered on one stream.
 *  - Checks the host can make (shapes, null pointers, 16-byte alignment of
 *    vector-loaded tensors, workspace size) return a negative NVQ_E* code and
 *    enqueue nothing.  A HIP launch failure returns NVQ_EHIP.
 *  - Conditions only the device sees set bits of a status word kept in the
 *    workspace (NVQ_STATUS_*), read with nvq_device_status().
 *  - bf16 tensors are passed as uint16_t bit patterns.
 *  - Empty inputs: a tensor whose row (or token) count is 0 may be passed as
 *    NULL.  The outputs that are not empty are still written as the
 *    definitions give them: nvfp4_quantize with rows == 0 writes
 *    s_t = fl32(amax / 2688) with the amax of nothing taken as 0 (or
 *    amax_in) and chan_score = 0; nvq_moe_permute with T == 0 writes all-zero
 *    expert offsets; the WGRAD mode of qat_fakequant_gemm_w4a16 writes dw = 0
 *    (leaves it with accumulate) for experts without rows.
 */
#ifndef NVQ_H
#define NVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum nvq_status {
  NVQ_OK = 0,
  NVQ_EINVAL = -1,       /* null pointer or bad enum/value */
  NVQ_ESHAPE = -2,       /* shape not supported (K % 16, k > K, ...) */
  NVQ_EALIGN = -3,       /* a vector-loaded tensor is not 16-byte aligned */
  NVQ_EWORKSPACE = -4,   /* workspace missing or too small */
  NVQ_EHIP = -5,         /* a HIP runtime call failed */
  NVQ_EUNSUPPORTED = -6  /* valid request this build does not implement */
};

enum nvq_dtype { NVQ_F32 = 0, NVQ_BF16 = 1 };

/* device status bits (nvq_device_status) */
enum {
  NVQ_STATUS_NONFINITE = 1u << 0, /* a quantized input held Inf or NaN */
  NVQ_STATUS_BAD_EXPERT = 1u << 1, /* a top-k expert id was outside [0, E) */
  NVQ_STATUS_BAD_SLOT = 1u << 2,   /* a cache slot was past the last page */
  NVQ_STATUS_BAD_SEQUENCE = 1u << 3, /* a page id, length or row range of a sequence does not
                                       fit the cache, the block table or the query rows */
  NVQ_STATUS_BAD_TARGET = 1u << 4  /* a target was at or past the end of the vocabulary */
};

const char* nvq_status_string(int status);

/* Reads the status word of workspace `ws` after `stream` drains (this call
 * synchronizes the stream).  *flags receives NVQ_STATUS_* bits. */
int nvq_device_status(const void* ws, void* stream, uint32_t* flags);

/* ------------------------------------------------------------------------ */
/* NVFP4 quantization (QUADS §1, §2.1; TRACE "Fonctionnement").
 *
 * x        [batch, rows, K] of dtype x_dtype (NVQ_F32 or NVQ_BF16), 16-byte
 *          aligned; K % 16 == 0; 1 <= batch <= 65535.  Row r of item b starts
 *          at element (b * rows + r) * ldx: ldx >= K is the row stride in
 *          elements (0 means K, a dense tensor) and ldx * element size must be
 *          a multiple of 16 bytes (NVQ_EALIGN otherwise; ldx < K: NVQ_ESHAPE).
 *          Outputs are always dense.
 * amax_in  nullable device [batch] fp32: replaces amax_t = max|x| of each
 *          batch item (e.g. to requantize with a known scale).
 * codes    [batch, rows, K/2]  E2M1 codes, even element in the low nibble.
 * scales   [batch, rows, K/16] E4M3 block-scale codes (never 0x7F).
 * tensor_scale [batch] fp32 s_t = fl32(amax_t / 2688).
 * chan_score   nullable [K] fp32 (only with batch == 1): per-channel residual
 *          score, the sum of |x - dequant(q(x))| over rows in a fixed order
 *          (16-row sequential sub-chunk sums, summed in order within 128-row
 *          chunks, chunks summed in order; every sum fp32).
 * Decisions are exact: each scale is the E4M3 value nearest the real quotient
 * amax_b / (6 s_t) (ties to even, saturating at 448) and each code the E2M1
 * value nearest |x| / (s_b s_t) (ties to even, saturating at 6).
 * Each batch item is one tensor with its own s_t (stacked expert weights).
 * A non-finite input sets NVQ_STATUS_NONFINITE.
 */
size_t nvfp4_quantize_workspace_bytes(int64_t batch, int64_t rows, int64_t K);
int nvfp4_quantize(const void* x, int x_dtype, int64_t batch, int64_t rows, int64_t K,
                   int64_t ldx, const float* amax_in, uint8_t* codes, uint8_t* scales,
                   float* tensor_scale, float* chan_score, void* ws, size_t ws_bytes,
                   void* stream);

/* Allocation-free variant of nvfp4_quantize, for callers that cannot allocate
 * device memory or pass a workspace (code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation).  Same arguments, results
 * and host-side errors as nvfp4_quantize, without ws / ws_bytes: the scratch
 * memory (status word, amax partials, residual chunk partials) is a static
 * array inside the library, NVQ_QUANTIZE_NOALLOC_SCRATCH_BYTES on every GPU
 * the library runs on, held until the process ends.  A call whose scratch
 * need (nvfp4_quantize_workspace_bytes(batch, rows, K)) exceeds it returns
 * NVQ_EWORKSPACE and launches nothing.  The first call on a device looks up
 * that device's array (hipGetSymbolAddress); no call allocates.  Every call on
 * one GPU shares the array: calls that may overlap on one GPU (other streams,
 * other host threads) race and must be ordered by the caller.  The device
 * status word lives in the shared array and is not reported to the caller;
 * use nvfp4_quantize when NVQ_STATUS_NONFINITE must be read. */
#define NVQ_QUANTIZE_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
int nvfp4_quantize_noalloc(const void* x, int x_dtype, int64_t batch, int64_t rows, int64_t K,
                           int64_t ldx, const float* amax_in, uint8_t* codes, uint8_t* scales,
                           float* tensor_scale, float* chan_score, void* stream);

/* NVFP4 dequantization: y = sign * fl32(fl32(G * s_b) * s_t), written as fp32
 * (y_dtype NVQ_F32) or rounded to nearest-even bf16 (NVQ_BF16).  This is the
 * quantize-dequantize image both sides use for the weights (QUADS §2.1).
 * codes [batch, rows, K/2] (8-byte aligned), scales [batch, rows, K/16],
 * tensor_scale [batch], y [batch, rows, K] (16-byte aligned); K % 16 == 0,
 * 1 <= batch <= 65535.  No rows: nothing is written.  Errors (NVQ_EINVAL,
 * NVQ_ESHAPE, NVQ_EALIGN) launch nothing. */
int nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales, const float* tensor_scale,
                     int64_t batch, int64_t rows, int64_t K, void* y, int y_dtype, void* stream);

/* ------------------------------------------------------------------------ */
/* Rollout-guided rounding (TRACE post: "L'idée centrale de TRACE" -- the
 * rollout's quantization guides the trainer's rounding and the cache keeps
 * only the mantissa and the scale factors; "Fonctionnement, côté ingénierie"
 * -- each value rounds to the grid point above or below, the discrete choice
 * both sides must share).
 *
 * The guidance record of a quantized tensor is one bit per element, bits
 * [batch, rows, K/8] u8 (element c of a row in bit c % 8 of byte c / 8), kept
 * with the rollout's block scales and tensor scale: 0.1875 byte per element
 * against 0.5625 for codes + scales.
 *   NVQ_GUIDE_MANTISSA   the mantissa bit (index & 1) of the rollout's code;
 *   NVQ_GUIDE_DIRECTION  1 when the rollout's magnitude G s_b s_t lies strictly
 *                        above |x| (rounded up), else 0.
 */
enum { NVQ_GUIDE_MANTISSA = 0, NVQ_GUIDE_DIRECTION = 1 };

/* Writes the guidance record `bits` of the NVFP4 record (codes [batch, rows,
 * K/2], scales [batch, rows, K/16], tensor_scale [batch]) of x.  Mantissa mode
 * reads only the codes (x, scales, tensor_scale may be NULL); direction mode
 * reads x [batch, rows, K] (x_dtype NVQ_F32 or NVQ_BF16, 16-byte aligned), the
 * value that was quantized.  K % 16 == 0, 1 <= batch <= 65535; codes 8-byte
 * and bits 2-byte aligned.  Device pointers, caller-owned; asynchronous on stream.  Errors
 * (NVQ_EINVAL, NVQ_ESHAPE, NVQ_EALIGN) launch nothing. */
int nvfp4_guidance_record(const void* x, int x_dtype, const uint8_t* codes, const uint8_t* scales,
                          const float* tensor_scale, int64_t batch, int64_t rows, int64_t K,
                          int mode, uint8_t* bits, void* stream);

/* Rebuilds NVFP4 codes [batch, rows, K/2] for master values w [batch, rows, K]
 * (w_dtype NVQ_F32 or NVQ_BF16, e.g. weights the trainer has updated since the
 * rollout quantized them) from a guidance record: the rollout's scales
 * [batch, rows, K/16] and tensor_scale [batch] are reused unchanged, and for
 * each element, with lo / hi the indices of the grid points G s_b s_t at or
 * below / at or above |w| (hi = 7 beyond the grid):
 *   mantissa:  of a = min(lo, 6) and a + 1, the one whose mantissa bit is the
 *              recorded bit (adjacent E2M1 points differ in that bit);
 *   direction: recorded 1 -> hi, 0 -> lo.
 * The sign is signbit(w); a zero block or tensor scale gives magnitude 0.
 * Decisions are exact.  With w equal to the quantized tensor this gives back
 * the rollout's codes.  ws is nullable (else 256-byte aligned, >= 256 bytes):
 * a non-finite w sets NVQ_STATUS_NONFINITE in its status word (that element's
 * code is then unspecified).  K % 16 == 0, 1 <= batch <= 65535; w 16-byte,
 * codes 8-byte, bits 2-byte aligned.
 * Errors (NVQ_EINVAL, NVQ_ESHAPE, NVQ_EALIGN, NVQ_EWORKSPACE) launch nothing. */
int nvfp4_guided_quantize(const void* w, int w_dtype, int64_t batch, int64_t rows, int64_t K,
                          const uint8_t* bits, const uint8_t* scales, const float* tensor_scale,
                          int mode, uint8_t* codes, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Residual-channel selection (QUADS §2.2-B).
 *
 * Selects the k channels with the largest residual score (ties to the lower
 * channel index) and writes them in rank order to idx_out [k] (int32).
 * x [rows, K] (row stride ldx >= K elements, 0 means K) is the tensor whose
 * NVFP4 record (codes [rows, K/2], scales [rows, K/16], tensor_scale [1],
 * dense) is given; it is read only to recompute scores or residuals.
 * scores_in  nullable [K]: the chan_score of nvfp4_quantize.  When NULL the
 *            score is recomputed from x and its NVFP4 record (codes, scales,
 *            tensor_scale), in the same order as nvfp4_quantize.
 * scores_out nullable [K]: receives the score used.
 * resid_out  nullable [rows, k] bf16: the compensation operand
 *            bf16(fl32(x - dequant(q(x))))[:, idx_out].
 * 0 <= k <= K; k == 0 writes nothing to idx_out/resid_out.  k <= 1024 takes
 * any K (radix select); k > 1024 needs K <= 8192, else NVQ_EUNSUPPORTED.
 * Scores compare as numbers (-0 equals +0); they must not be NaN.
 */
size_t residual_topk_workspace_bytes(int64_t rows, int64_t K, int32_t k);
int residual_topk_channels(const void* x, int x_dtype, int64_t rows, int64_t K, int64_t ldx,
                           const uint8_t* codes, const uint8_t* scales,
                           const float* tensor_scale, const float* scores_in, float* scores_out,
                           int32_t k, int32_t* idx_out, uint16_t* resid_out, void* ws,
                           size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* MoE routing glue (TRACE "Fonctionnement": the router's discrete expert
 * choice).  Per token: the topk largest of E fp32 logits, descending, ties
 * to the lower expert id; weights = softmax over the chosen logits.
 * logits [T, E] fp32; ids [T, topk] int32; weights [T, topk] fp32.
 * Requires 1 <= topk <= E <= 1024. */
int nvq_moe_route(const float* logits, int64_t T, int64_t E, int64_t topk, int32_t* ids,
                  float* weights, void* stream);

/* Token-expert pairs p = t*topk + j sorted stably by expert (histogram,
 * exclusive scan, stable scatter).  ids [T, topk]; sorted_pair [P];
 * expert_offsets [E+1] (rows of expert e are [off[e], off[e+1])); pos [P]
 * the inverse map (sorted position of pair p).  An id outside [0, E) sets
 * NVQ_STATUS_BAD_EXPERT and that pair is dropped. */
size_t nvq_moe_permute_workspace_bytes(int64_t T, int64_t topk, int64_t E);
int nvq_moe_permute(const int32_t* ids, int64_t T, int64_t topk, int64_t E,
                    int32_t* sorted_pair, int32_t* expert_offsets, int32_t* pos, void* ws,
                    size_t ws_bytes, void* stream);

/* out[t, n] = bf16( sum_j w[t, j] * y[pos[t*topk + j], n] ), j ascending, fp32
 * accumulation.  y [P, N] bf16 in sorted-pair order; a pair the permutation
 * dropped (pos < 0) is left out of the sum.  N % 8 == 0.
 * out_amax: nullable device fp32 word (4-byte aligned) that receives max |out|
 * over the stored bf16 values (0 for no tokens); the call clears it first.
 * When out is the next layer's input (QUADS §2.1: activations are quantized
 * online at every forward), passing it as amax_in to nvfp4_quantize replaces
 * that call's amax pass with an identical result.  Calls sharing the word
 * must be ordered on one stream. */
int nvq_moe_combine(const uint16_t* y, const int32_t* pos, const float* weights, int64_t T,
                    int64_t topk, int64_t N, uint16_t* out, float* out_amax, void* stream);

/* ------------------------------------------------------------------------ */
/* Chained backward of the MoE layer's glue (QUADS §2.2-A: the trainer's
 * backward with the identity straight-through estimator runs through the
 * layer's SwiGLU and expert combine; its GEMMs are qat_fakequant_gemm_w4a16).
 * All tensors bf16 unless stated, row-major, 16-byte aligned device pointers,
 * caller-owned; asynchronous on stream; errors (NVQ_EINVAL, NVQ_ESHAPE,
 * NVQ_EALIGN) launch nothing.  Zero rows (tokens) do nothing. */

/* h [rows, I] = bf16(silu(g) u) with g = y1[:, :I], u = y1[:, I:], y1
 * [rows, 2I] of dtype y1_dtype (NVQ_F32 or NVQ_BF16), silu(g) = g / (1 +
 * exp(-g)), evaluated in fp32 with the hardware exp and reciprocal (the
 * result is rounded to bf16).  I % 8 == 0. */
int nvq_swiglu_forward(const void* y1, int y1_dtype, int64_t rows, int64_t I, uint16_t* h,
                       void* stream);

/* dy1 [rows, 2I] = (dh u s (1 + g (1 - s)), dh g s), s = 1 / (1 + exp(-g)):
 * the gradient of h = silu(g) u with respect to the gate and up
 * pre-activations y1 (layout and dtype as above), given dh [rows, I].  fp32
 * arithmetic, bf16 result.  I % 8 == 0. */
int nvq_swiglu_backward(const void* y1, int y1_dtype, const uint16_t* dh, int64_t rows, int64_t I,
                        uint16_t* dy1, void* stream);

/* Backward of nvq_moe_combine (out[t] = sum_j w[t,j] y[pos[t,j]]):
 *   dy[pos[t,j], :] = bf16(fl32(w[t,j] dout[t, :]))   dy [P, N] sorted-pair order
 *   dw[t, j]       = sum_n dout[t,n] y[pos[t,j], n]   fp32 (nullable; y is read
 *                    only for it)
 * dout [T, N]; pos [T, topk] the permutation's inverse map (pairs with pos < 0
 * are skipped, their dw is 0); weights [T, topk] fp32.  N % 8 == 0.  The token
 * gradient of the gate/up input, sum_j dx_pairs[pos[t,j]], is nvq_moe_combine
 * with unit weights. */
int nvq_moe_combine_backward(const uint16_t* dout, const uint16_t* y, const int32_t* pos,
                             const float* weights, int64_t T, int64_t topk, int64_t N,
                             uint16_t* dy, float* dw, void* stream);

/* ------------------------------------------------------------------------ */
/* W4A4 MoE grouped GEMM with residual compensation (QUADS §1, §2.2-B).
 *
 * For every sorted row p of expert e (off[e] <= p < off[e+1]) and t = a_row[p]:
 *   Y[p, n] = s_tA s_tW sum_c G_A[t,c] s_bA[t,c] G_W[e,n,c] s_bW[e,n,c]
 *           + s_tW sum_j resid[t, j] G_W[e,n,idx_j] s_bW[e,n,idx_j]
 * i.e. deq(qA) deq(qW_e)^T plus the bf16 residual of the selected channels
 * times the dequantized weight columns.  fp32 accumulation.
 * Epilogue NVQ_EPI_NONE writes Y (bf16 [rows, N] and/or fp32 [rows, N]);
 * NVQ_EPI_SWIGLU writes h = bf16(silu(Y[:, :N/2]) * Y[:, N/2:]) [rows, N/2]
 * (out_f32, if given, still receives the full pre-activation Y).
 * Path NVQ_GEMM_DEQ16 (what NVQ_GEMM_AUTO selects) dequantizes each NVFP4 tile
 * exactly to fp16 and feeds fp16 MFMA, in 128-row tiles; NVQ_GEMM_DEQ16_WIDE
 * is the same arithmetic in 256-row tiles with both operands dequantized once
 * per workgroup (an evaluated alternative; slower here).  NVQ_GEMM_FP8_BLOCK
 * runs one FP8 MFMA per
 * 16-element block on the raw E2M1 magnitudes and applies both block scales to
 * the block product in fp32 (the evaluated alternative; same result to
 * rounding, slower).  K % 128 == 0; k % 8 == 0. */
enum { NVQ_EPI_NONE = 0, NVQ_EPI_SWIGLU = 1 };
enum { NVQ_GEMM_AUTO = 0, NVQ_GEMM_DEQ16 = 1, NVQ_GEMM_FP8_BLOCK = 2, NVQ_GEMM_DEQ16_WIDE = 3 };

typedef struct nvq_moe_gemm_args {
  size_t struct_size;            /* sizeof(nvq_moe_gemm_args) */
  int64_t rows;                  /* P: sorted rows */
  int64_t K, N, E;
  int64_t a_rows;                /* rows of the A record (tokens) */
  const int32_t* a_row;          /* [rows] A row of each sorted row; NULL = identity */
  const int32_t* expert_offsets; /* [E+1] */
  const uint8_t* a_codes;        /* [a_rows, K/2] */
  const uint8_t* a_scales;       /* [a_rows, K/16] */
  const float* a_tensor_scale;   /* [1] */
  const uint16_t* a_resid;       /* [a_rows, k] bf16 compensation operand (k > 0) */
  const int32_t* comp_idx;       /* [k] selected channels */
  int32_t k;                     /* multiple of 8; 0 disables the compensation */
  const uint8_t* w_codes;        /* [E, N, K/2] */
  const uint8_t* w_scales;       /* [E, N, K/16] */
  const float* w_tensor_scale;   /* [E] */
  int32_t epilogue;
  int32_t path;
  uint16_t* out_bf16;            /* [rows, N] or [rows, N/2] (SWIGLU); nullable if out_f32 */
  float* out_f32;                /* [rows, N] fp32 pre-epilogue; nullable */
  void* ws;
  size_t ws_bytes;
  int32_t a_row_div;             /* > 0: A row of sorted row p is a_row[p] / a_row_div
                                    (pass sorted pair ids with topk); 0: a_row[p] */
  /* Optional, read only when struct_size covers them: the channel-major copy of
   * the weight record made by nvfp4_channel_major.  When both are set the
   * compensation columns are gathered from it (the k selected channels are k
   * contiguous rows there) instead of from every row of w_codes. */
  const uint8_t* w_codes_cm;     /* [E, K, N/2] or NULL */
  const uint8_t* w_scales_cm;    /* [E, K/16, N] or NULL */
  /* Optional, read only when struct_size covers it: with NVQ_EPI_SWIGLU, a
   * device fp32 word (4-byte aligned) that receives max |h| over every row
   * the call writes, taken on the stored bf16 values (the call clears it
   * first; 0 for no rows).  Passed as amax_in to nvfp4_quantize of h, it
   * replaces that call's own amax pass with an identical result (a maximum
   * does not depend on order).  NULL: not computed.  NVQ_EINVAL with another
   * epilogue.  Calls sharing the word must be ordered on one stream. */
  float* h_amax;
  /* Optional, read only when struct_size covers them: the layer's combine
   * fused into this call (NVQ_EPI_NONE, path DEQ16 or AUTO; out_bf16 needed):
   * comb_out[t, n] = bf16( sum_j comb_weights[t, j] * out_bf16[comb_pos[t*topk
   * + j], n] ), j ascending, fp32 -- the same values as nvq_moe_combine on this
   * call's bf16 output, bit for bit (QUADS §2.2-B asks for the correction in
   * fused kernels).  comb_pair [rows] is the sorted pair id of each row (token
   * = pair / comb_topk), comb_pos [comb_T, comb_topk] the permutation's inverse
   * map (pos < 0: dropped pair), comb_weights [comb_T, comb_topk].  Each output
   * row piece is written by the last workgroup to finish a row of that token
   * (arrival counters in the workspace; moe_gemm_workspace_bytes_comb).
   * comb_out NULL: no combine. */
  const int32_t* comb_pair;
  const int32_t* comb_pos;
  const float* comb_weights;
  int64_t comb_T;
  int32_t comb_topk;
  uint16_t* comb_out;
} nvq_moe_gemm_args;

/* Channel-major copy of an NVFP4 weight record (same codes and scales, other
 * layout), for the compensation gather of moe_grouped_gemm_w4a4_comp: the
 * correction multiplies the residual by the weight columns of the selected
 * channels (QUADS §2.2-B), and in the row-major record one column touches
 * every weight row.  Built once per weight version (the rollout's weights are
 * static between syncs).
 *   codes  [batch, N, K/2] (even element in the low nibble) -> codes_cm [batch, K, N/2]
 *          (row n even in the low nibble)
 *   scales [batch, N, K/16]                                -> scales_cm [batch, K/16, N]
 * N % 16 == 0, K % 16 == 0, 1 <= batch <= 65535; codes and codes_cm 8-byte
 * aligned.  Device pointers, caller-owned, no overlap; asynchronous on stream.
 * Errors: NVQ_EINVAL (null pointer), NVQ_ESHAPE, NVQ_EALIGN; nothing is
 * launched then. */
int nvfp4_channel_major(const uint8_t* codes, const uint8_t* scales, int64_t batch, int64_t N,
                        int64_t K, uint8_t* codes_cm, uint8_t* scales_cm, void* stream);

/* Workspace: tile table plus the packed compensation weights [E, N, k16] bf16;
 * the _comb variant also holds the fused combine's arrival counters (T tokens). */
size_t moe_gemm_workspace_bytes(int64_t rows, int64_t E, int64_t N, int32_t k);
size_t moe_gemm_workspace_bytes_comb(int64_t rows, int64_t E, int64_t N, int32_t k, int64_t T);
int moe_grouped_gemm_w4a4_comp(const nvq_moe_gemm_args* args, void* stream);

/* ------------------------------------------------------------------------ */
/* Asymmetric W4A16 QAT grouped GEMMs (QUADS §2.2-A; TRACE "L'idée centrale"):
 * the weight is the dequantized NVFP4 record W^_e = deq(codes, scales, s_t)
 * taken as-is from the rollout (its rounding is reused, not recomputed);
 * activations stay bf16.  Identity straight-through gradient.
 *   FWD   y[p, n]  = sum_c x[a_row[p], c] W^_e[n, c]        -> [rows, N]
 *   DGRAD dx[p, c] = sum_n dy[p, n] W^_e[n, c]              -> [rows, K]
 *   WGRAD dw[e, n, c] (+)= sum_{p of e} dy[p, n] x[a_row[p], c]  -> [E, N, K] fp32
 * fp32 accumulation. */
enum { NVQ_QAT_FWD = 0, NVQ_QAT_DGRAD = 1, NVQ_QAT_WGRAD = 2 };

typedef struct nvq_qat_gemm_args {
  size_t struct_size;            /* sizeof(nvq_qat_gemm_args) */
  int32_t mode;
  int32_t accumulate;            /* WGRAD: 1 adds to dw, 0 overwrites */
  int64_t rows, K, N, E;
  int64_t x_rows;
  const int32_t* a_row;          /* [rows] row of x for each sorted row; NULL = identity */
  const int32_t* expert_offsets; /* [E+1] */
  const uint16_t* x;             /* [x_rows, K] bf16 (FWD, WGRAD) */
  const uint16_t* dy;            /* [rows, N] bf16 (DGRAD, WGRAD) */
  const uint8_t* w_codes;        /* [E, N, K/2] */
  const uint8_t* w_scales;       /* [E, N, K/16] */
  const float* w_tensor_scale;   /* [E] */
  uint16_t* out_bf16;            /* FWD y / DGRAD dx, nullable if out_f32 */
  float* out_f32;                /* FWD y / DGRAD dx fp32, nullable */
  float* dw;                     /* WGRAD [E, N, K] */
  void* ws;
  size_t ws_bytes;
} nvq_qat_gemm_args;

size_t qat_gemm_workspace_bytes(int64_t rows, int64_t E);
int qat_fakequant_gemm_w4a16(const nvq_qat_gemm_args* args, void* stream);

/* ------------------------------------------------------------------------ */
/* Rotary positions of projected heads (the step before the FP4 KV cache of
 * the rollout, TRACE "Résultats"; the gradient is the trainer's side of it).
 *
 * Token t, head h, pair j of rot_dim / 2, angle a = positions[t] * inv_freq[j]:
 *   y_u = m (x_u cos a - x_w sin a),  y_w = m (x_u sin a + x_w cos a)
 * with (u, w) = (j, j + rot_dim / 2) for NVQ_ROPE_HALF and (2j, 2j + 1) for
 * NVQ_ROPE_INTERLEAVED; elements at or past rot_dim are copied.  inverse != 0
 * turns by -a with the same m: the gradient of the forward call.
 *
 * x, y      [T, H, D] of dtype NVQ_F32 or NVQ_BF16, unit element stride; token
 *           t, head h of x starts at element t * x_ld_t + h * x_ld_h (0 means
 *           dense: H * D and D), of y likewise.  y == x with equal strides
 *           works in place (then elements past rot_dim are not touched); any
 *           other overlap is not supported.  No alignment beyond the element's
 *           is required; 16-byte aligned rows with rot_dim % 16 == 0 (bf16) or
 *           % 8 (fp32), D a multiple of 8 (bf16) or 4, take the vector path.
 * positions [T] int32, any value.  inv_freq [rot_dim / 2] fp64, radians per
 *           position.  Angles are reduced in fp64 (for frequencies up to 1
 *           their error stays below 2^-20 radians at every int32 position),
 *           sine, cosine and the products are fp32, rounded once to dtype.
 * 2 <= rot_dim <= D <= 4096, rot_dim even, H <= 65535, T < 2^24; the
 * rows of y do not overlap.
 * Asynchronous on stream; errors (NVQ_EINVAL, NVQ_ESHAPE, NVQ_EALIGN) launch
 * nothing; T == 0 or H == 0 does nothing. */
enum { NVQ_ROPE_HALF = 0, NVQ_ROPE_INTERLEAVED = 1 };
int nvq_rope(const void* x, int dtype, int64_t T, int64_t H, int64_t D, int64_t x_ld_t,
             int64_t x_ld_h, const int32_t* positions, const double* inv_freq, int64_t rot_dim,
             int layout, float magnitude, int inverse, void* y, int64_t y_ld_t, int64_t y_ld_h,
             void* stream);

/* Frequencies of the rotation, written to HOST memory: inv_freq [rot_dim / 2]
 * fp64 with f_j = base^(-2j / rot_dim), stretched for long contexts by kind:
 *   NVQ_ROPE_PLAIN   f_j
 *   NVQ_ROPE_LINEAR  f_j / factor (positions divided by factor)
 *   NVQ_ROPE_BASE    f_j of the base base * factor^(rot_dim / (rot_dim - 2)),
 *                    which leaves the fastest pair and divides the slowest by
 *                    factor (rot_dim > 2)
 *   NVQ_ROPE_RAMP    r f_j + (1 - r) f_j / factor, r = clamp((n_j - slow) /
 *                    (fast - slow), 0, 1) with n_j = orig_len f_j / (2 pi) the
 *                    pair's turns over the original context (0 < slow < fast);
 *                    *magnitude = 0.1 ln(factor) + 1.
 * The ramp is linear in the pairs' turns.  A checkpoint that was stretched with
 * another ramp (one linear in the pair index, say) brings its own inv_freq.
 * *magnitude (nullable) is 1 for the other kinds.  factor >= 1, base > 0 (> 1
 * for NVQ_ROPE_BASE).  No HIP call.  NVQ_EINVAL / NVQ_ESHAPE. */
enum { NVQ_ROPE_PLAIN = 0, NVQ_ROPE_LINEAR = 1, NVQ_ROPE_BASE = 2, NVQ_ROPE_RAMP = 3 };
int nvq_rope_frequencies(int kind, int64_t rot_dim, double base, double factor, double orig_len,
                         double slow, double fast, double* inv_freq, float* magnitude);

/* ------------------------------------------------------------------------ */
/* Paged NVFP4 KV cache (TRACE "Résultats": FP4 weights, activations and KV
 * cache in the rollout).
 *
 * One layer's K and V as two NVFP4 records with 16-element blocks along the
 * head dimension and one static tensor scale each, in num_pages pages of
 * page_size slots.  Slot s is offset s % page_size of page s / page_size; the
 * slots of one (page, head) are contiguous.  V keeps its block scales with
 * the slots innermost, because attention contracts over the slots there: the
 * scales of one block of consecutive keys come with one load.
 * All buffers are device memory of the caller; codes and k_scales, v_scales
 * 16-byte aligned.  page_size is a power of two, 16 <= page_size <= 65536;
 * head_dim % 16 == 0, 16 <= head_dim <= 512; 1 <= heads <= 65535;
 * num_pages >= 1.  Contents never written may hold any bytes. */
typedef struct nvq_kv_cache {
  size_t struct_size;          /* sizeof(nvq_kv_cache) */
  uint8_t* k_codes;            /* [num_pages, heads, page_size, head_dim / 2] */
  uint8_t* k_scales;           /* [num_pages, heads, page_size, head_dim / 16] */
  uint8_t* v_codes;            /* [num_pages, heads, page_size, head_dim / 2] */
  uint8_t* v_scales;           /* [num_pages, heads, head_dim / 16, page_size] */
  const float* k_tensor_scale; /* [1] s_t of K (amax / 2688) */
  const float* v_tensor_scale; /* [1] s_t of V */
  int64_t num_pages;
  int32_t page_size, heads, head_dim;
} nvq_kv_cache;

/* Quantizes T new tokens as it writes them: k and v [T, heads, head_dim] of
 * dtype NVQ_F32 or NVQ_BF16 (token t, head h at element t * ld_t + h * ld_h, 0
 * meaning dense; rows 16-byte aligned) go to slots[t].  The bytes are those of
 * nvfp4_quantize with the cache's tensor scales (exact decisions; values past
 * 2688 s_t saturate).  A negative slot skips the token; a slot past the last
 * page skips it and sets NVQ_STATUS_BAD_SLOT; a non-finite value sets
 * NVQ_STATUS_NONFINITE (its block is unspecified).  Slots that no token names
 * keep their bytes.  The slots of one call should differ: where two tokens
 * name one slot, each of its bytes is one of theirs.
 * ws nullable (else 256-byte aligned, >= 256 bytes): receives the status word.
 * T < 2^24; num_pages * page_size <= INT32_MAX.  Asynchronous on stream;
 * errors (NVQ_EINVAL, NVQ_ESHAPE, NVQ_EALIGN, NVQ_EWORKSPACE) launch nothing. */
int nvq_kv_append(const nvq_kv_cache* cache, const void* k, const void* v, int dtype, int64_t T,
                  int64_t k_ld_t, int64_t k_ld_h, int64_t v_ld_t, int64_t v_ld_h,
                  const int32_t* slots, void* ws, size_t ws_bytes, void* stream);

/* Reads T slots back: k_out and v_out [T, heads, head_dim] dense, of dtype
 * out_dtype, receive sign * fl32(fl32(G s_b) s_t) (rounded to nearest-even for
 * NVQ_BF16), as nvfp4_dequantize gives it.  Either output may be NULL; they
 * are 16-byte aligned.  A negative slot gives zeros; a slot past the last
 * page gives zeros and sets NVQ_STATUS_BAD_SLOT.  A slot may be read any
 * number of times.  ws and limits as for nvq_kv_append. */
int nvq_kv_gather(const nvq_kv_cache* cache, const int32_t* slots, int64_t T, void* k_out,
                  void* v_out, int out_dtype, void* ws, size_t ws_bytes, void* stream);

/* Attention of a chunk of new tokens over the paged cache, for single decoded
 * tokens, drafted tokens and prompt chunks alike.
 *
 * Sequence b owns the query rows cu_q[b] .. cu_q[b + 1] - 1 and the keys 0 ..
 * kv_len[b] - 1; key j lies in slot j % page_size of page block_table[b,
 * j / page_size].  Row i of its n is at position p = kv_len[b] - n + i (the
 * new tokens are the last ones, already appended).  Query head h reads
 * key/value head h / (q_heads / heads).  With K^, V^ the dequantized record:
 *   out[row, h] = sum_j w_j V^[j],  w = softmax_j(softmax_scale q . K^[j])
 * over the visible keys: j <= p if causal (every key of the sequence if not),
 * and j > p - window if window > 0 (causal only).  A row without visible keys
 * gives zeros and lse = -inf.  lse [total_q, q_heads] (nullable) receives the
 * natural logarithm of the sum of exponentials.
 * q is bf16.  For head dimensions 64, 128 and 256 it is held in fp16 under a
 * power of two per row and head, which is exact for elements down to 2^-31 of
 * the largest and off by at most 2^-39 of it for smaller ones; q . K^ is summed
 * in fp32 from exact products, the softmax is fp32, its weights are rounded to
 * fp16 for the product with V^ (2^-11 relative), out is rounded to bf16.  Other
 * head dimensions keep q and the weights in fp32.  A query that holds a NaN
 * gives NaN, out and lse, if its row sees a key; scores of -inf weigh nothing,
 * and a row that has no others counts as one without visible keys.
 *
 * Rows that no sequence owns (before cu_q[0], from cu_q[B] on) are not
 * written.  A page id outside [0, num_pages), keys past the block table's
 * width, kv_len < 0, a decreasing or too large cu_q, or more than max_q rows
 * in a sequence set NVQ_STATUS_BAD_SEQUENCE in the workspace's status word:
 * such keys are left out, a negative length counts as 0, ranges are cut to
 * [0, total_q] and rows past the max_q-th are not written.  No call reads or
 * writes outside its buffers for any content of the index arrays.  Sequences
 * may share pages.  out may be q with the same strides; it overlaps nothing else
 * of the call.  Calls on one stream may share a workspace. */
typedef struct nvq_paged_attention_args {
  size_t struct_size;          /* sizeof(nvq_paged_attention_args) */
  int64_t total_q, B;          /* query rows; sequences */
  int64_t max_q;               /* no sequence has more new tokens; 0: total_q.  It and the table's
                                  width choose the kernels: values near the batch's own are faster */
  int32_t q_heads;             /* a multiple of cache->heads */
  int32_t causal;              /* 0 or 1 */
  int64_t window;              /* 0: none */
  float softmax_scale;
  const uint16_t* q;           /* [total_q, q_heads, head_dim] bf16, 16-byte aligned rows */
  int64_t q_ld_t, q_ld_h;      /* strides in elements; 0: dense */
  const int32_t* cu_q;         /* [B + 1] */
  const int32_t* kv_len;       /* [B] */
  const int32_t* block_table;  /* [B, table_width], row stride table_ld (0: table_width) */
  int64_t table_width, table_ld;
  uint16_t* out;               /* [total_q, q_heads, head_dim] bf16, 16-byte aligned rows */
  int64_t out_ld_t, out_ld_h;
  float* lse;                  /* [total_q, q_heads] fp32 or NULL */
  void* ws;                    /* 256-byte aligned */
  size_t ws_bytes;
} nvq_paged_attention_args;

/* Workspace of a call with these arguments (only the sizes are read: total_q,
 * B, max_q, q_heads, window, table_width and the cache's heads, head_dim,
 * page_size). */
size_t nvq_paged_attention_workspace_bytes(const nvq_kv_cache* cache,
                                           const nvq_paged_attention_args* args);
/* Limits: total_q < 2^24, q_heads <= 32768, total_q * q_heads <= 2^30, B <=
 * 65535, B * heads <= 2^21, B * table_width <= 2^30, table_width * page_size <= INT32_MAX,
 * B * (table_width * page_size / 128 + 2) <= INT32_MAX.
 * Errors: NVQ_EINVAL, NVQ_ESHAPE, NVQ_EALIGN, NVQ_EWORKSPACE; nothing is
 * launched then. */
int nvq_paged_attention(const nvq_kv_cache* cache, const nvq_paged_attention_args* args,
                        void* stream);

/* ------------------------------------------------------------------------ */
/* What a trainer runs around its QAT layers (QUADS §2.2-A: the optimizer
 * updates the master weights after every step; §2.1: both sides compare the
 * log-probabilities of sampled tokens): the norm in front of a layer, the loss
 * at the model's end, the gradient norm before the optimizer. */

/* RMS norm with the residual's addition:
 *   h = x + residual, rounded to their type (x itself without a residual)
 *   y = h weight r,  r = (mean of h^2 over the row + eps)^(-1/2)
 * The sum of squares is fp64, r and the products fp32, y is rounded once.
 * x, residual, h, y  [T, D] of dtype NVQ_F32 or NVQ_BF16, row strides in
 *   elements (0: D), rows 16-byte aligned.  h is written only with a residual
 *   (required then) and may be x or residual with the same stride; so may y, but
 *   it may not be h too (NVQ_EINVAL).
 * weight  [D] of w_dtype (either type), 16-byte aligned.
 * y8      nullable [T, D] E4M3 codes (8-byte aligned), dense, with y8_scales fp32
 *   [T, D / group], or [T] for group == 0 (one scale a row): scale = max|y| of
 *   the group / 448 in fp32 (at least 2^-126), code = the E4M3 value nearest the
 *   real quotient 448 y / max|y|, ties to even (exact decisions).  group is 0,
 *   32, 64 or 128 and divides D.  A group that holds a NaN has a NaN scale and
 *   NaN codes (0x7F or 0xFF).
 * y and y8 may both be given; one must be.
 * rstd    nullable [T] fp32: r, for the gradient.
 * out_amax nullable fp32 word, needs y: max |y| over the stored values (the
 *   call clears it first), as amax_in of nvfp4_quantize it replaces that
 *   call's amax pass with an identical result.  Calls sharing the word must
 *   be ordered on one stream.
 * 8 <= D <= 32768, D % 8 == 0; T < 2^24; eps >= 0.  No workspace.  T == 0
 * clears out_amax and does nothing else.  Asynchronous on stream; errors
 * (NVQ_EINVAL, NVQ_ESHAPE, NVQ_EALIGN) launch nothing. */
typedef struct nvq_rms_norm_args {
  size_t struct_size;          /* sizeof(nvq_rms_norm_args) */
  int64_t T, D;
  int32_t dtype, w_dtype;
  const void* x;
  int64_t x_ld;
  const void* residual;        /* nullable */
  int64_t res_ld;
  const void* weight;
  double eps;
  void* h;
  int64_t h_ld;
  void* y;
  int64_t y_ld;
  uint8_t* y8;
  float* y8_scales;
  int32_t group;
  float* rstd;
  float* out_amax;
} nvq_rms_norm_args;
int nvq_rms_norm(const nvq_rms_norm_args* args, void* stream);

/* Gradient of nvq_rms_norm, with u = h rstd and g = dy weight:
 *   dx      = rstd (g - u mean(g u)) + dh    the same for x and the residual
 *   dweight = (old +) sum over rows of dy u  fp32, in a fixed order
 * dy, h, dh, dx [T, D] of dtype (strides and alignment as above); dh, the
 * gradient that reaches h from elsewhere (the residual stream), is nullable; h
 * is what the forward call wrote (x without a residual), rstd [T] its r.  dx
 * may be dy, h or dh with the same stride.  dweight is nullable [D] fp32, added
 * to with accumulate; only it needs the workspace (no status word is kept).
 * fp32 arithmetic.  Limits and errors as above, and NVQ_EWORKSPACE. */
typedef struct nvq_rms_norm_grad_args {
  size_t struct_size;          /* sizeof(nvq_rms_norm_grad_args) */
  int64_t T, D;
  int32_t dtype, w_dtype;
  const void* dy;
  int64_t dy_ld;
  const void* h;
  int64_t h_ld;
  const void* weight;
  const float* rstd;
  const void* dh;
  int64_t dh_ld;
  void* dx;
  int64_t dx_ld;
  float* dweight;
  int32_t accumulate;
  void* ws;
  size_t ws_bytes;
} nvq_rms_norm_grad_args;
size_t nvq_rms_norm_backward_workspace_bytes(int64_t T, int64_t D);
int nvq_rms_norm_backward(const nvq_rms_norm_grad_args* args, void* stream);

/* Linear cross entropy: the softmax cross entropy of z = scale x w^T against
 * the targets, without keeping z.  Per token t:
 *   lse[t]  = ln sum_v exp z[t, v]
 *   loss[t] = lse[t] - z[t, targets[t]], minus the target's log-probability
 * x [T, D] and w [V, D] bf16, row strides in elements (0: D), rows 16-byte
 * aligned; targets [T] int32.  A negative target (padding) has loss 0; one >= V
 * too, and sets NVQ_STATUS_BAD_TARGET.  lse is written for every token.
 * loss is the target's distance from the largest logit and what the others add
 * to it, not the difference of two large numbers: it is never negative.
 * Products are summed in fp32, exponentials and sums are fp32.  A token with a
 * NaN or +inf logit has NaN results; logits of -inf weigh nothing.
 * loss and lse [T] fp32, each nullable (not both).
 *
 * The gradient, given lse and dloss [T] fp32 (NULL: 1 for every token):
 *   c[t, v] = exp(z[t, v] - lse[t]) - [v = targets[t]]
 *   dx[t] = scale dloss[t] sum_v c[t, v] w[v]   bf16 [T, D], nullable, stride dx_ld
 *   dw[v] = scale sum_t c[t, v] dloss[t] x[t]   [V, D] of dw_dtype (NVQ_BF16 or
 *           NVQ_F32), nullable, stride dw_ld; added to with accumulate
 * Tokens without a valid target or with dloss == 0 do not count: their dx is 0
 * and nothing they hold reaches dw.  c times the mantissa of dloss over the
 * largest finite |dloss| is computed in fp32 and rounded to bf16 (at most 2^-8
 * relative for each entry; powers of two of the weights are exact, and where
 * weights are not a power of two apart, what a target's own terms of dx and dw
 * lose is added again: they are good to 2^-15); all sums are fp32, dx and dw are
 * rounded once.  dx and dw overlap
 * nothing else of the call.  Results do not depend on the order in which
 * workgroups run.
 * 8 <= D <= 65536, D % 8 == 0; 1 <= V <= 2^24; T <= 2^23; T V <= 2^39 (each
 * rounded up to 256); strides of x and w at most 2^21.  T == 0 writes dw = 0
 * (leaves it with accumulate).  The gradient's workspace holds a piece of c (at
 * most 2^28 entries, or 256 words of the vocabulary for every token), the states
 * of the tokens that count twice (as they are, and weighted), and dx in fp32.
 * Asynchronous on stream; errors (NVQ_EINVAL, NVQ_ESHAPE, NVQ_EALIGN,
 * NVQ_EWORKSPACE) launch nothing. */
typedef struct nvq_linear_ce_args {
  size_t struct_size;          /* sizeof(nvq_linear_ce_args) */
  int64_t T, D, V;
  const uint16_t* x;
  int64_t x_ld;
  const uint16_t* w;
  int64_t w_ld;
  const int32_t* targets;
  float scale;
  float* loss;                 /* forward only */
  float* lse;                  /* forward: out; gradient: in */
  const float* dloss;          /* gradient only, like what follows */
  uint16_t* dx;
  int64_t dx_ld;
  void* dw;
  int64_t dw_ld;
  int32_t dw_dtype, accumulate;
  void* ws;
  size_t ws_bytes;
} nvq_linear_ce_args;
size_t nvq_linear_cross_entropy_workspace_bytes(int64_t T, int64_t D, int64_t V);
int nvq_linear_cross_entropy(const nvq_linear_ce_args* args, void* stream);
size_t nvq_linear_cross_entropy_backward_workspace_bytes(int64_t T, int64_t D, int64_t V);
int nvq_linear_cross_entropy_backward(const nvq_linear_ce_args* args, void* stream);

/* Tensors of one call: arrays in HOST memory, read before the call returns.
 * data[i] is a device pointer to numel[i] dense elements of dtype[i] (NVQ_F32
 * or NVQ_BF16), aligned to its element (16-byte alignment is faster);
 * 0 <= numel <= 2^42; count <= 2^20. */
typedef struct nvq_tensor_list {
  size_t struct_size;          /* sizeof(nvq_tensor_list) */
  int64_t count;
  void* const* data;
  const int64_t* numel;
  const int32_t* dtype;
} nvq_tensor_list;

/* norm[0] (fp32, device) = sqrt(sum of squares over all elements of grads),
 * squares and sums fp64 in a fixed order.  nvq_clip_grad_norm also writes
 *   out_i = grads_i min(1, max_norm / norm)
 * rounded to its type: in place with out == NULL (gradients within max_norm
 * are then not touched), else into tensors of the same sizes and types.  A
 * norm[0] that is not finite (one past the largest fp32 number too) scales
 * nothing (out receives the gradients bit by bit) and sets
 * NVQ_STATUS_NONFINITE.  max_norm >= 0; infinity never clips.  Tensors that are
 * written overlap no other of the call (NVQ_EINVAL), but out_i may be grads_i.  A
 * captured graph keeps the tensors' addresses.  Asynchronous on stream; errors
 * (NVQ_EINVAL, NVQ_ESHAPE, NVQ_EALIGN, NVQ_EWORKSPACE) launch nothing. */
size_t nvq_grad_norm_workspace_bytes(const nvq_tensor_list* grads);
int nvq_grad_norm(const nvq_tensor_list* grads, float* norm, void* ws, size_t ws_bytes, void* stream);
int nvq_clip_grad_norm(const nvq_tensor_list* grads, const nvq_tensor_list* out, float max_norm,
                       float* norm, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVQ_H */
