"""Thin Python binding of libnvq.so (include/nvq.h): argument marshalling only.

torch provides device memory and the current HIP stream; every step of the
computation runs in the library's HIP kernels.  There is no CPU fallback: if
the library is missing or the device is not a GPU, calls raise.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvq.so")

NVQ_F32, NVQ_BF16 = 0, 1
NVQ_EPI_NONE, NVQ_EPI_SWIGLU = 0, 1
NVQ_GEMM_AUTO, NVQ_GEMM_DEQ16, NVQ_GEMM_FP8_BLOCK, NVQ_GEMM_DEQ16_WIDE = 0, 1, 2, 3
NVQ_QAT_FWD, NVQ_QAT_DGRAD, NVQ_QAT_WGRAD = 0, 1, 2
NVQ_STATUS_NONFINITE, NVQ_STATUS_BAD_EXPERT = 1, 2
NVQ_STATUS_BAD_SLOT, NVQ_STATUS_BAD_SEQUENCE = 4, 8
NVQ_GUIDE_MANTISSA, NVQ_GUIDE_DIRECTION = 0, 1
NVQ_ROPE_HALF, NVQ_ROPE_INTERLEAVED = 0, 1
NVQ_ROPE_PLAIN, NVQ_ROPE_LINEAR, NVQ_ROPE_BASE, NVQ_ROPE_RAMP = 0, 1, 2, 3

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t

_lock = threading.Lock()
_lib = None


class NvqError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {code} ({status_string(code)})")
        self.code = code


class MoeGemmArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", _SZ), ("rows", _I64), ("K", _I64), ("N", _I64), ("E", _I64),
        ("a_rows", _I64), ("a_row", _P), ("expert_offsets", _P), ("a_codes", _P),
        ("a_scales", _P), ("a_tensor_scale", _P), ("a_resid", _P), ("comp_idx", _P),
        ("k", _I32), ("w_codes", _P), ("w_scales", _P), ("w_tensor_scale", _P),
        ("epilogue", _I32), ("path", _I32), ("out_bf16", _P), ("out_f32", _P),
        ("ws", _P), ("ws_bytes", _SZ), ("a_row_div", _I32), ("w_codes_cm", _P),
        ("w_scales_cm", _P), ("h_amax", _P), ("comb_pair", _P), ("comb_pos", _P),
        ("comb_weights", _P), ("comb_T", _I64), ("comb_topk", _I32), ("comb_out", _P),
    ]


class QatGemmArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", _SZ), ("mode", _I32), ("accumulate", _I32), ("rows", _I64), ("K", _I64),
        ("N", _I64), ("E", _I64), ("x_rows", _I64), ("a_row", _P), ("expert_offsets", _P),
        ("x", _P), ("dy", _P), ("w_codes", _P), ("w_scales", _P), ("w_tensor_scale", _P),
        ("out_bf16", _P), ("out_f32", _P), ("dw", _P), ("ws", _P), ("ws_bytes", _SZ),
    ]


class KvCacheArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", _SZ), ("k_codes", _P), ("k_scales", _P), ("v_codes", _P), ("v_scales", _P),
        ("k_tensor_scale", _P), ("v_tensor_scale", _P), ("num_pages", _I64), ("page_size", _I32),
        ("heads", _I32), ("head_dim", _I32),
    ]


class PagedAttentionArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", _SZ), ("total_q", _I64), ("B", _I64), ("max_q", _I64), ("q_heads", _I32),
        ("causal", _I32), ("window", _I64), ("softmax_scale", ctypes.c_float), ("q", _P),
        ("q_ld_t", _I64), ("q_ld_h", _I64), ("cu_q", _P), ("kv_len", _P), ("block_table", _P),
        ("table_width", _I64), ("table_ld", _I64), ("out", _P), ("out_ld_t", _I64),
        ("out_ld_h", _I64), ("lse", _P), ("ws", _P), ("ws_bytes", _SZ),
    ]


# (name, restype, argtypes)
_SIGS = [
    ("nvq_status_string", ctypes.c_char_p, [ctypes.c_int]),
    ("nvq_device_status", ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_uint32)]),
    ("nvfp4_quantize_workspace_bytes", _SZ, [_I64, _I64, _I64]),
    ("nvfp4_quantize", ctypes.c_int,
     [_P, ctypes.c_int, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    ("nvfp4_quantize_noalloc", ctypes.c_int,
     [_P, ctypes.c_int, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P]),
    ("nvfp4_dequantize", ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _P, ctypes.c_int, _P]),
    ("nvfp4_guidance_record", ctypes.c_int,
     [_P, ctypes.c_int, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, _P, _P]),
    ("nvfp4_guided_quantize", ctypes.c_int,
     [_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, _P, ctypes.c_int, _P, _P, _SZ, _P]),
    ("residual_topk_workspace_bytes", _SZ, [_I64, _I64, _I32]),
    ("residual_topk_channels", ctypes.c_int,
     [_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _SZ, _P]),
    ("nvq_moe_route", ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _P]),
    ("nvq_moe_permute_workspace_bytes", _SZ, [_I64, _I64, _I64]),
    ("nvq_moe_permute", ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _SZ, _P]),
    ("nvq_moe_combine", ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _P, _P, _P]),
    ("nvq_swiglu_forward", ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _P, _P]),
    ("nvq_swiglu_backward", ctypes.c_int, [_P, ctypes.c_int, _P, _I64, _I64, _P, _P]),
    ("nvq_moe_combine_backward", ctypes.c_int, [_P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P]),
    ("nvfp4_channel_major", ctypes.c_int, [_P, _P, _I64, _I64, _I64, _P, _P, _P]),
    ("moe_gemm_workspace_bytes", _SZ, [_I64, _I64, _I64, _I32]),
    ("moe_gemm_workspace_bytes_comb", _SZ, [_I64, _I64, _I64, _I32, _I64]),
    ("moe_grouped_gemm_w4a4_comp", ctypes.c_int, [ctypes.POINTER(MoeGemmArgs), _P]),
    ("qat_gemm_workspace_bytes", _SZ, [_I64, _I64]),
    ("qat_fakequant_gemm_w4a16", ctypes.c_int, [ctypes.POINTER(QatGemmArgs), _P]),
    ("nvq_rope", ctypes.c_int,
     [_P, ctypes.c_int, _I64, _I64, _I64, _I64, _I64, _P, _P, _I64, ctypes.c_int, ctypes.c_float,
      ctypes.c_int, _P, _I64, _I64, _P]),
    ("nvq_rope_frequencies", ctypes.c_int,
     [ctypes.c_int, _I64] + [ctypes.c_double] * 5 + [_P, ctypes.POINTER(ctypes.c_float)]),
    ("nvq_kv_append", ctypes.c_int,
     [ctypes.POINTER(KvCacheArgs), _P, _P, ctypes.c_int, _I64, _I64, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    ("nvq_kv_gather", ctypes.c_int,
     [ctypes.POINTER(KvCacheArgs), _P, _I64, _P, _P, ctypes.c_int, _P, _SZ, _P]),
    ("nvq_paged_attention_workspace_bytes", _SZ, [ctypes.POINTER(KvCacheArgs), _P]),
    ("nvq_paged_attention", ctypes.c_int, [ctypes.POINTER(KvCacheArgs), _P, _P]),
]

EXPORTED = [s[0] for s in _SIGS]


def load(path: str = LIB_PATH):
    """Load libnvq.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with `python -m qat_nvfp4_quantize_amd.build`")
            L = ctypes.CDLL(path)
            for name, res, args in _SIGS:
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def status_string(code: int) -> str:
    try:
        return load().nvq_status_string(code).decode()
    except Exception:  # pragma: no cover
        return "?"


def _check(fn, rc):
    if rc != 0:
        raise NvqError(fn, rc)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _dev_rows(t, name):
    """A GPU tensor whose rows may be strided: [rows, K] or [batch, rows, K]
    with unit element stride and (for 3-D) items rows * ldx elements apart.
    Returns ldx, the row stride in elements."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() not in (2, 3) or t.stride(-1) != 1:
        raise ValueError(f"{name} must be [rows, K] or [batch, rows, K] with unit column stride")
    rows, K = t.shape[-2], t.shape[-1]
    many = t.dim() == 3 and t.shape[0] > 1
    if rows > 1:
        ldx = t.stride(-2)
    else:  # one row per item: the item stride is the row stride
        ldx = t.stride(0) if many else K
    if many and t.stride(0) != rows * ldx:
        raise ValueError(f"{name}: batch items must be rows * ldx elements apart")
    return ldx


def _dtype_code(t):
    if t.dtype == torch.float32:
        return NVQ_F32
    if t.dtype == torch.bfloat16:
        return NVQ_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


def workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def device_status(ws: torch.Tensor) -> int:
    v = ctypes.c_uint32(0)
    _check("nvq_device_status", load().nvq_device_status(_ptr(ws), _stream(), ctypes.byref(v)))
    return v.value


# ----------------------------------------------------------------- quantize --
def nvfp4_quantize(x, amax_in=None, score=False, ws=None, out=None):
    """NVFP4-quantize x [rows, K] or [batch, rows, K] (fp32/bf16); rows may be
    strided (a column slice of a wider tensor).

    Returns (codes u8 [..., K/2], scales u8 [..., K/16], tensor_scale f32 [batch],
    score f32 [K] or None, ws)."""
    ldx = _dev_rows(x, "x")
    L = load()
    batch, rows, K = (1, *x.shape) if x.dim() == 2 else tuple(x.shape)
    lead = x.shape[:-1]
    if out is None:
        codes = torch.empty(*lead, K // 2, dtype=torch.uint8, device=x.device)
        scales = torch.empty(*lead, K // 16, dtype=torch.uint8, device=x.device)
        st = torch.empty(batch, dtype=torch.float32, device=x.device)
        sc = torch.empty(K, dtype=torch.float32, device=x.device) if score else None
    else:
        codes, scales, st, sc = out
    if ws is None:
        ws = workspace(L.nvfp4_quantize_workspace_bytes(batch, rows, K), x.device)
    if amax_in is not None:
        _dev(amax_in, "amax_in")
    rc = L.nvfp4_quantize(_ptr(x), _dtype_code(x), batch, rows, K, ldx, _ptr(amax_in),
                          _ptr(codes), _ptr(scales), _ptr(st), _ptr(sc), _ptr(ws), ws.numel(),
                          _stream())
    _check("nvfp4_quantize", rc)
    return codes, scales, st, sc, ws


NVQ_QUANTIZE_NOALLOC_SCRATCH_BYTES = 16 << 20


def nvfp4_quantize_noalloc(x, amax_in=None, score=False, out=None):
    """nvfp4_quantize without a workspace: the library's static per-device
    scratch serves the call (calls on one GPU must not overlap).  Returns
    (codes, scales, tensor_scale, score or None)."""
    ldx = _dev_rows(x, "x")
    batch, rows, K = (1, *x.shape) if x.dim() == 2 else tuple(x.shape)
    lead = x.shape[:-1]
    if out is None:
        codes = torch.empty(*lead, K // 2, dtype=torch.uint8, device=x.device)
        scales = torch.empty(*lead, K // 16, dtype=torch.uint8, device=x.device)
        st = torch.empty(batch, dtype=torch.float32, device=x.device)
        sc = torch.empty(K, dtype=torch.float32, device=x.device) if score else None
    else:
        codes, scales, st, sc = out
    if amax_in is not None:
        _dev(amax_in, "amax_in")
    rc = load().nvfp4_quantize_noalloc(_ptr(x), _dtype_code(x), batch, rows, K, ldx,
                                       _ptr(amax_in), _ptr(codes), _ptr(scales), _ptr(st),
                                       _ptr(sc), _stream())
    _check("nvfp4_quantize_noalloc", rc)
    return codes, scales, st, sc


def nvfp4_dequantize(codes, scales, tensor_scale, out_dtype=torch.float32, batch=None, out=None):
    _dev(codes, "codes")
    K = codes.shape[-1] * 2
    if batch is None:
        batch = tensor_scale.numel()
    rows = codes.numel() // (K // 2) // batch
    y = out if out is not None else torch.empty(*codes.shape[:-1], K, dtype=out_dtype,
                                                device=codes.device)
    rc = load().nvfp4_dequantize(_ptr(codes), _ptr(scales), _ptr(tensor_scale), batch, rows, K,
                                 _ptr(y), _dtype_code(y), _stream())
    _check("nvfp4_dequantize", rc)
    return y


def _batch_rows(t, per_row, batch):
    """(batch, rows) of a [rows, n] or [batch, rows, n] tensor."""
    if batch is None:
        batch = t.shape[0] if t.dim() == 3 else 1
    return batch, t.numel() // per_row // batch


def nvfp4_guidance_record(codes, mode, x=None, scales=None, tensor_scale=None, batch=None,
                          out=None):
    """TRACE guidance record of an NVFP4 record: bits u8 [..., K/8].  Mantissa
    mode needs only the codes; direction mode needs x (the quantized values),
    scales and tensor_scale."""
    _dev(codes, "codes")
    K = codes.shape[-1] * 2
    batch, rows = _batch_rows(codes, K // 2, batch)
    bits = out if out is not None else torch.empty(
        *codes.shape[:-1], K // 8, dtype=torch.uint8, device=codes.device)
    xd = _dtype_code(x) if x is not None else NVQ_F32
    rc = load().nvfp4_guidance_record(_ptr(x), xd, _ptr(codes), _ptr(scales), _ptr(tensor_scale),
                                      batch, rows, K, mode, _ptr(bits), _stream())
    _check("nvfp4_guidance_record", rc)
    return bits


def nvfp4_guided_quantize(w, bits, scales, tensor_scale, mode, ws=None, out=None):
    """Codes u8 [..., K/2] of master values w rebuilt from a guidance record
    (bits, the rollout's scales and tensor scales).  ws (optional, >= 256
    bytes) receives the non-finite status bit."""
    _dev(w, "w")
    K = w.shape[-1]
    batch, rows = _batch_rows(w, K, None)
    codes = out if out is not None else torch.empty(
        *w.shape[:-1], K // 2, dtype=torch.uint8, device=w.device)
    rc = load().nvfp4_guided_quantize(_ptr(w), _dtype_code(w), batch, rows, K, _ptr(bits),
                                      _ptr(scales), _ptr(tensor_scale), mode, _ptr(codes),
                                      _ptr(ws), 0 if ws is None else ws.numel(), _stream())
    _check("nvfp4_guided_quantize", rc)
    return codes


def residual_topk_channels(x, codes, scales, tensor_scale, k, scores=None, want_scores=False,
                           want_resid=True, ws=None):
    """Returns (idx int32 [k], resid bf16 [rows, k] or None, scores f32 [K] or None).
    x [rows, K] may have strided rows."""
    ldx = _dev_rows(x, "x")
    L = load()
    rows, K = x.shape
    idx = torch.empty(max(k, 1), dtype=torch.int32, device=x.device)
    resid = torch.empty(rows, max(k, 1), dtype=torch.bfloat16, device=x.device) if want_resid else None
    sc_out = torch.empty(K, dtype=torch.float32, device=x.device) if want_scores else None
    if ws is None:
        ws = workspace(L.residual_topk_workspace_bytes(rows, K, k), x.device)
    rc = L.residual_topk_channels(_ptr(x), _dtype_code(x), rows, K, ldx, _ptr(codes), _ptr(scales),
                                  _ptr(tensor_scale), _ptr(scores), _ptr(sc_out), k, _ptr(idx),
                                  _ptr(resid), _ptr(ws), ws.numel(), _stream())
    _check("residual_topk_channels", rc)
    return idx[:k], (resid[:, :k] if resid is not None else None), sc_out


# ---------------------------------------------------------------- MoE glue --
def nvq_moe_route(logits, topk):
    _dev(logits, "logits")
    T, E = logits.shape
    ids = torch.empty(T, topk, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, topk, dtype=torch.float32, device=logits.device)
    _check("nvq_moe_route", load().nvq_moe_route(_ptr(logits), T, E, topk, _ptr(ids), _ptr(w),
                                                 _stream()))
    return ids, w


def nvq_moe_permute(ids, E, ws=None):
    _dev(ids, "ids")
    L = load()
    T, topk = ids.shape
    P = T * topk
    sp = torch.empty(P, dtype=torch.int32, device=ids.device)
    off = torch.empty(E + 1, dtype=torch.int32, device=ids.device)
    pos = torch.empty(P, dtype=torch.int32, device=ids.device)
    if ws is None:
        ws = workspace(L.nvq_moe_permute_workspace_bytes(T, topk, E), ids.device)
    _check("nvq_moe_permute", L.nvq_moe_permute(_ptr(ids), T, topk, E, _ptr(sp), _ptr(off),
                                                _ptr(pos), _ptr(ws), ws.numel(), _stream()))
    return sp, off, pos, ws


def nvq_moe_combine(y, pos, weights, out=None, out_amax=None):
    """out bf16 [T, N]; out_amax (optional fp32 [1] on the GPU) receives max |out|."""
    _dev(y, "y")
    T, topk = weights.shape
    N = y.shape[1]
    if out is None:
        out = torch.empty(T, N, dtype=torch.bfloat16, device=y.device)
    _check("nvq_moe_combine", load().nvq_moe_combine(_ptr(y), _ptr(pos), _ptr(weights), T, topk,
                                                     N, _ptr(out), _ptr(out_amax), _stream()))
    return out


def nvq_swiglu_forward(y1, out=None):
    """h bf16 [rows, I] = silu(y1[:, :I]) * y1[:, I:] (y1 fp32 or bf16 [rows, 2I])."""
    _dev(y1, "y1")
    rows, two_i = y1.shape
    h = out if out is not None else torch.empty(rows, two_i // 2, dtype=torch.bfloat16,
                                                device=y1.device)
    _check("nvq_swiglu_forward", load().nvq_swiglu_forward(_ptr(y1), _dtype_code(y1), rows,
                                                           two_i // 2, _ptr(h), _stream()))
    return h


def nvq_swiglu_backward(y1, dh, out=None):
    """dy1 bf16 [rows, 2I]: gradient of h = silu(g) u w.r.t. (g, u) given dh."""
    _dev(y1, "y1")
    _dev(dh, "dh")
    rows, two_i = y1.shape
    dy1 = out if out is not None else torch.empty(rows, two_i, dtype=torch.bfloat16,
                                                  device=y1.device)
    _check("nvq_swiglu_backward", load().nvq_swiglu_backward(
        _ptr(y1), _dtype_code(y1), _ptr(dh), rows, two_i // 2, _ptr(dy1), _stream()))
    return dy1


def nvq_moe_combine_backward(dout, pos, weights, rows, y=None, want_dw=True, out=None):
    """(dy bf16 [rows, N] in sorted-pair order, dw fp32 [T, topk] or None)."""
    _dev(dout, "dout")
    T, N = dout.shape
    topk = weights.shape[1]
    if out is not None:
        dy, dw = out
    else:
        dy = torch.empty(rows, N, dtype=torch.bfloat16, device=dout.device)
        dw = torch.empty(T, topk, dtype=torch.float32, device=dout.device) if want_dw else None
    _check("nvq_moe_combine_backward", load().nvq_moe_combine_backward(
        _ptr(dout), _ptr(y), _ptr(pos), _ptr(weights), T, topk, N, _ptr(dy), _ptr(dw), _stream()))
    return dy, dw


# ------------------------------------------------------------------- GEMMs --
def nvfp4_channel_major(codes, scales, out=None):
    """Channel-major copy of a weight record: codes [B, N, K/2] -> [B, K, N/2],
    scales [B, N, K/16] -> [B, K/16, N].  Returns (codes_cm, scales_cm)."""
    _dev(codes, "codes")
    L = load()
    if codes.dim() == 2:
        codes, scales = codes.unsqueeze(0), scales.unsqueeze(0)
    B, N, Kh = codes.shape
    K = Kh * 2
    if out is None:
        out = (torch.empty(B, K, N // 2, dtype=torch.uint8, device=codes.device),
               torch.empty(B, K // 16, N, dtype=torch.uint8, device=codes.device))
    _check("nvfp4_channel_major",
           L.nvfp4_channel_major(_ptr(codes), _ptr(scales), B, N, K, _ptr(out[0]), _ptr(out[1]),
                                 _stream()))
    return out


def moe_grouped_gemm_w4a4_comp(a_codes, a_scales, a_tensor_scale, w_codes, w_scales,
                               w_tensor_scale, expert_offsets, rows, a_row=None, a_resid=None,
                               comp_idx=None, epilogue=NVQ_EPI_NONE, path=NVQ_GEMM_AUTO,
                               want_bf16=True, want_f32=False, ws=None, a_row_div=0, out=None,
                               w_cm=None, h_amax=None, comb=None):
    """Returns (out_bf16 or None, out_f32 or None).  w_cm: optional
    (codes_cm, scales_cm) from nvfp4_channel_major for the compensation gather.
    comb: optional (sorted_pair, pos, weights, out) -- the layer's combine fused
    into this call, written to out bf16 [T, N]."""
    L = load()
    E, N, Kh = w_codes.shape
    K = Kh * 2
    dev = w_codes.device
    k = 0 if comp_idx is None else int(comp_idx.numel())
    n_out = N // 2 if epilogue == NVQ_EPI_SWIGLU else N
    if out is not None:
        ob, of = out
    else:
        ob = torch.empty(rows, n_out, dtype=torch.bfloat16, device=dev) if want_bf16 else None
        of = torch.empty(rows, N, dtype=torch.float32, device=dev) if want_f32 else None
    if ws is None:
        if comb is None:
            ws = workspace(L.moe_gemm_workspace_bytes(rows, E, N, k), dev)
        else:
            ws = workspace(L.moe_gemm_workspace_bytes_comb(rows, E, N, k, comb[2].shape[0]), dev)
    a = MoeGemmArgs()
    a.struct_size = ctypes.sizeof(MoeGemmArgs)
    a.rows, a.K, a.N, a.E = rows, K, N, E
    a.a_rows = a_codes.shape[0]
    a.a_row = _ptr(a_row)
    a.expert_offsets = _ptr(expert_offsets)
    a.a_codes, a.a_scales, a.a_tensor_scale = _ptr(a_codes), _ptr(a_scales), _ptr(a_tensor_scale)
    a.a_resid = _ptr(a_resid)
    a.comp_idx = _ptr(comp_idx)
    a.k = k
    a.w_codes, a.w_scales, a.w_tensor_scale = _ptr(w_codes), _ptr(w_scales), _ptr(w_tensor_scale)
    a.epilogue, a.path = epilogue, path
    a.out_bf16, a.out_f32 = _ptr(ob), _ptr(of)
    a.ws, a.ws_bytes = _ptr(ws), ws.numel()
    a.a_row_div = int(a_row_div)
    if w_cm is not None:
        a.w_codes_cm, a.w_scales_cm = _ptr(w_cm[0]), _ptr(w_cm[1])
    a.h_amax = _ptr(h_amax)
    if comb is not None:
        sp, pos, wts, cout = comb
        a.comb_pair, a.comb_pos, a.comb_weights = _ptr(sp), _ptr(pos), _ptr(wts)
        a.comb_T, a.comb_topk = wts.shape[0], wts.shape[1]
        a.comb_out = _ptr(cout)
    _check("moe_grouped_gemm_w4a4_comp", L.moe_grouped_gemm_w4a4_comp(ctypes.byref(a), _stream()))
    return ob, of


def qat_fakequant_gemm_w4a16(mode, w_codes, w_scales, w_tensor_scale, expert_offsets, rows,
                             x=None, dy=None, a_row=None, dw=None, accumulate=False,
                             want_bf16=True, want_f32=False, ws=None, out=None):
    """FWD: returns (y_bf16, y_f32); DGRAD: (dx_bf16, dx_f32); WGRAD: dw [E, N, K] fp32."""
    L = load()
    E, N, Kh = w_codes.shape
    K = Kh * 2
    dev = w_codes.device
    ob = of = None
    if mode in (NVQ_QAT_FWD, NVQ_QAT_DGRAD):
        cols = N if mode == NVQ_QAT_FWD else K
        if out is not None:
            ob, of = out
        else:
            ob = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev) if want_bf16 else None
            of = torch.empty(rows, cols, dtype=torch.float32, device=dev) if want_f32 else None
    elif dw is None:
        dw = torch.empty(E, N, K, dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(L.qat_gemm_workspace_bytes(rows, E), dev)
    a = QatGemmArgs()
    a.struct_size = ctypes.sizeof(QatGemmArgs)
    a.mode, a.accumulate = mode, int(bool(accumulate))
    a.rows, a.K, a.N, a.E = rows, K, N, E
    a.x_rows = 0 if x is None else x.shape[0]
    a.a_row = _ptr(a_row)
    a.expert_offsets = _ptr(expert_offsets)
    a.x, a.dy = _ptr(x), _ptr(dy)
    a.w_codes, a.w_scales, a.w_tensor_scale = _ptr(w_codes), _ptr(w_scales), _ptr(w_tensor_scale)
    a.out_bf16, a.out_f32 = _ptr(ob), _ptr(of)
    a.dw = _ptr(dw)
    a.ws, a.ws_bytes = _ptr(ws), ws.numel()
    _check("qat_fakequant_gemm_w4a16", L.qat_fakequant_gemm_w4a16(ctypes.byref(a), _stream()))
    if mode == NVQ_QAT_WGRAD:
        return dw
    return ob, of


# ------------------------------------------ rotary positions, paged KV cache --
# A decode step makes these calls for every layer, and their kernels run for a
# few microseconds, so the checks below are kept to attribute reads.
_HEAD_TYPES = (torch.bfloat16, torch.float32)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(fn, name, dev, *args):
    """Calls the library with `dev` as the current device, on its current stream."""
    index = dev.index
    if _current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != 0:
        raise NvqError(name, rc)


def _on(dev, **tensors):
    """Raises for the first tensor that does not lie on the GPU `dev`."""
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be a GPU tensor on {dev}, got {t.device}")


def _ws_args(ws):
    """(pointer, bytes) of a workspace, which the library writes from its start
    to its end: a tensor of any type and shape without gaps, or None."""
    if ws is None:
        return None, 0
    if not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous, got {list(ws.shape)}, strides {list(ws.stride())}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _typed(t, name, dtype, *shape):
    """A contiguous tensor of this dtype and (where given) shape."""
    if t.dtype != dtype or not t.is_contiguous() or (shape and t.shape != shape):
        raise ValueError(f"{name} must be contiguous {dtype}" + (f" {list(shape)}" if shape else "")
                         + f", got {t.dtype} {list(t.shape)}, strides {list(t.stride())}")


def _heads(t, name, dtypes=_HEAD_TYPES):
    """(T, H, D, ld_t, ld_h) of [T, H, D] projected heads with unit element
    stride, tokens and heads strided freely (a slice of a fused projection);
    a stride of 0 stands for the dense one, also where the axis has one entry."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != 3 or t.dtype not in dtypes:
        raise ValueError(f"{name} must be [T, H, D] of {dtypes}, got {t.dtype} {list(t.shape)}")
    T, H, D = t.shape
    if t.is_contiguous():
        return T, H, D, 0, 0
    st, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (T > 1 and st <= 0) or (H > 1 and sh <= 0):
        raise ValueError(f"{name} must have unit element stride and no broadcast axis, got "
                         f"strides {t.stride()}")
    return T, H, D, (st if T > 1 else 0), (sh if H > 1 else 0)


def nvq_rope_frequencies(rot_dim, base=10000.0, kind=NVQ_ROPE_PLAIN, factor=1.0, orig_len=0.0,
                         slow=1.0, fast=32.0):
    """(inv_freq fp64 [rot_dim / 2] on the CPU, magnitude): the rotation's
    radians a position, stretched for long contexts by kind."""
    f = torch.empty(max(int(rot_dim), 0) // 2, dtype=torch.float64)
    m = ctypes.c_float(1.0)
    _check("nvq_rope_frequencies", load().nvq_rope_frequencies(
        kind, rot_dim, base, factor, orig_len, slow, fast, f.data_ptr() or None, ctypes.byref(m)))
    return f, m.value


def nvq_rope(x, positions, inv_freq, interleaved=False, magnitude=1.0, inverse=False, out=None):
    """x [T, H, D] (bf16/fp32, tokens and heads may be strided) with the first
    2 * len(inv_freq) elements of each head turned by positions [T] int32 times
    inv_freq (fp64, on the GPU); inverse turns back (the gradient).  out: a
    tensor like x to write, x itself for in place.  Like every call here it is
    not recorded for autograd: the gradient is the inverse call."""
    T, H, D, ld_t, ld_h = _heads(x, "x")
    dev = x.device
    old_t = old_h = 0
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        if out.shape != x.shape or out.dtype != x.dtype:
            raise ValueError("out must have the shape and dtype of x")
        _, _, _, old_t, old_h = _heads(out, "out")
    _typed(positions, "positions", torch.int32, T)
    _typed(inv_freq, "inv_freq", torch.float64)
    _on(dev, positions=positions, inv_freq=inv_freq, out=out)
    _call((_lib or load()).nvq_rope, "nvq_rope", dev, x.data_ptr(), _dtype_code(x), T, H, D, ld_t, ld_h,
          positions.data_ptr(), inv_freq.data_ptr(), 2 * inv_freq.numel(), 1 if interleaved else 0,
          magnitude, 1 if inverse else 0, out.data_ptr(), old_t, old_h)
    return out


class KvCache:
    """The paged NVFP4 cache of one layer over the caller's buffers: k_codes,
    v_codes u8 [pages, heads, page_size, D/2], k_scales u8 [pages, heads,
    page_size, D/16], v_scales u8 [pages, heads, D/16, page_size], and the
    tensor scales k_scale, v_scale fp32 [1]."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_scale, v_scale):
        if not k_codes.is_cuda or k_codes.dim() != 4:
            raise ValueError("k_codes must be a GPU tensor [pages, heads, page_size, D/2]")
        P, H, S, half = k_codes.shape
        D = 2 * half
        _typed(k_codes, "k_codes", torch.uint8)
        _typed(v_codes, "v_codes", torch.uint8, P, H, S, half)
        _typed(k_scales, "k_scales", torch.uint8, P, H, S, D // 16)
        _typed(v_scales, "v_scales", torch.uint8, P, H, D // 16, S)
        _typed(k_scale, "k_scale", torch.float32, 1)
        _typed(v_scale, "v_scale", torch.float32, 1)
        self.device = k_codes.device
        _on(self.device, k_scales=k_scales, v_codes=v_codes, v_scales=v_scales, k_scale=k_scale,
            v_scale=v_scale)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_scale, self.v_scale = k_scale, v_scale
        self.num_pages, self.heads, self.page_size, self.head_dim = P, H, S, D
        self.args = KvCacheArgs(ctypes.sizeof(KvCacheArgs), k_codes.data_ptr(), k_scales.data_ptr(),
                                v_codes.data_ptr(), v_scales.data_ptr(), k_scale.data_ptr(),
                                v_scale.data_ptr(), P, S, H, D)
        self._ref = ctypes.byref(self.args)

    @classmethod
    def empty(cls, num_pages, heads, page_size, head_dim, k_amax, v_amax, device="cuda"):
        """A cache of uninitialised pages whose tensor scales are calibrated to
        the given amax values (s_t = amax / 2688)."""
        def u8(*shape):
            return torch.empty(num_pages, heads, *shape, dtype=torch.uint8, device=device)

        # the fp32 quotient of nvfp4_quantize: rounded once from fp64
        st = (torch.tensor([k_amax, v_amax], dtype=torch.float32).double() / 2688.0).float().to(device)
        return cls(u8(page_size, head_dim // 2), u8(page_size, head_dim // 16),
                   u8(page_size, head_dim // 2), u8(head_dim // 16, page_size), st[0:1].clone(),
                   st[1:2].clone())


def nvq_kv_append(cache, k, v, slots, ws=None):
    """Quantizes the new tokens k, v [T, heads, D] (bf16/fp32, tokens and heads
    may be strided) into the cache's slots [T] int32 (page * page_size + offset,
    negative: skipped).  Bad slots and non-finite values raise nothing: they
    show in device_status(ws) of a caller's ws (>= 256 bytes)."""
    T, H, D, k_t, k_h = _heads(k, "k")
    _, _, _, v_t, v_h = _heads(v, "v")
    if k.shape != v.shape or k.dtype != v.dtype or H != cache.heads or D != cache.head_dim:
        raise ValueError(f"k and v must be [T, {cache.heads}, {cache.head_dim}] of one dtype, got "
                         f"{k.dtype} {list(k.shape)} and {v.dtype} {list(v.shape)}")
    _typed(slots, "slots", torch.int32, T)
    _on(cache.device, k=k, v=v, slots=slots, ws=ws)
    _call((_lib or load()).nvq_kv_append, "nvq_kv_append", cache.device, cache._ref, k.data_ptr(),
          v.data_ptr(), _dtype_code(k), T, k_t, k_h, v_t, v_h, slots.data_ptr(), *_ws_args(ws))


def nvq_kv_gather(cache, slots, out_dtype=torch.bfloat16, out=None, ws=None):
    """(k, v) [T, heads, D] read back from the cache's slots [T] int32 (a
    negative slot: zeros).  Bad slots raise nothing (zeros): they show in
    device_status(ws) of a caller's ws (>= 256 bytes)."""
    T = slots.numel()
    _typed(slots, "slots", torch.int32, T)
    shape = (T, cache.heads, cache.head_dim)
    if out is None:
        if out_dtype not in _HEAD_TYPES:
            raise ValueError(f"unsupported dtype {out_dtype}")
        k, v = torch.empty((2, *shape), dtype=out_dtype, device=cache.device).unbind(0)
    else:
        k, v = out
        _typed(k, "k", k.dtype, *shape)
        _typed(v, "v", k.dtype, *shape)
    _on(cache.device, slots=slots, k=k, v=v, ws=ws)
    _call((_lib or load()).nvq_kv_gather, "nvq_kv_gather", cache.device, cache._ref, slots.data_ptr(), T,
          k.data_ptr(), v.data_ptr(), _dtype_code(k), *_ws_args(ws))
    return k, v


def nvq_paged_attention(q, cache, cu_q, kv_len, block_table, max_q=None, scale=None, causal=True,
                        window=0, lse=None, out=None, ws=None):
    """Attention of the new tokens q [total_q, q_heads, D] (bf16, tokens and
    heads may be strided) over the cache: sequence b owns rows cu_q[b] ..
    cu_q[b + 1] - 1 and keys 0 .. kv_len[b] - 1, in the pages block_table[b].
    cu_q [B + 1], kv_len [B], block_table [B, width] int32 (rows may be
    strided).  max_q: no sequence has more new tokens (default: total_q, which
    plans a decode batch like prompts: pass 1 there).  scale defaults to D^-1/2.
    lse: optional fp32 [total_q, q_heads] to receive the log-sum-exp.  ws: a
    workspace to reuse (default: one for the call).  Returns out, bf16 like q.

    Rows that no sequence owns (padding before cu_q[0] or from cu_q[B] on, and a
    sequence's rows past max_q) are not written: without `out` they hold
    whatever the allocation did.  Mistakes in the index arrays raise nothing:
    they set a bit that only device_status(ws) of a caller's ws shows."""
    T, Hq, D, ld_t, ld_h = _heads(q, "q", (torch.bfloat16,))
    dev = cache.device
    if D != cache.head_dim:
        raise ValueError(f"q must have the cache's head_dim {cache.head_dim}, got {D}")
    B = kv_len.numel()
    _typed(cu_q, "cu_q", torch.int32, B + 1)
    _typed(kv_len, "kv_len", torch.int32, B)
    if block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.shape[0] != B:
        raise ValueError(f"block_table must be int32 [{B}, width]")
    width = table_ld = block_table.shape[1]
    if not block_table.is_contiguous():
        table_ld, unit = block_table.stride()
        if B == 1:
            table_ld = width
        if (width > 1 and unit != 1) or table_ld < width:
            raise ValueError("block_table must have unit column stride and rows that do not overlap")
    o_t = o_h = 0
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        _, _, _, o_t, o_h = _heads(out, "out", (torch.bfloat16,))
    if lse is not None:
        _typed(lse, "lse", torch.float32, T, Hq)
    _on(dev, q=q, cu_q=cu_q, kv_len=kv_len, block_table=block_table, out=out, lse=lse, ws=ws)
    head = (_ATTENTION.size, T, B, 0 if max_q is None else max_q, Hq, 1 if causal else 0, window,
            D ** -0.5 if scale is None else scale, q.data_ptr(), ld_t, ld_h, cu_q.data_ptr(),
            kv_len.data_ptr(), block_table.data_ptr(), width, table_ld, out.data_ptr(), o_t, o_h,
            0 if lse is None else lse.data_ptr())
    L = _lib or load()
    if ws is None:
        args = _ATTENTION.pack(*head, 0, 0)
        if _current_device() == dev.index:
            nbytes = L.nvq_paged_attention_workspace_bytes(cache._ref, args)
        else:
            with torch.cuda.device(dev):
                nbytes = L.nvq_paged_attention_workspace_bytes(cache._ref, args)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _call(L.nvq_paged_attention, "nvq_paged_attention", dev, cache._ref,
          _ATTENTION.pack(*head, *_ws_args(ws)))
    return out


# nvq_paged_attention_args as bytes: packing them takes a fifth of the time that
# filling a ctypes structure does, which a decode step would notice
_ATTENTION = struct.Struct("@Nqqqiiqf4xPqqPPPqqPqqPPN")
assert _ATTENTION.size == ctypes.sizeof(PagedAttentionArgs)
