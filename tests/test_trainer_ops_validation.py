"""Arguments that the norm, the loss and the clipping refuse, before anything
is launched (no GPU: the pointers are never followed)."""
import ctypes

import pytest

from qat_nvfp4_quantize_amd import nvq

OK_PTR = 0x100000
EINVAL, ESHAPE, EALIGN, EWORKSPACE = -1, -2, -3, -4


def _lib():
    import os

    if not os.path.exists(nvq.LIB_PATH):
        pytest.skip("libnvq.so not built")
    return nvq.load()


def _norm(**kw):
    a = nvq.RmsNormArgs(struct_size=ctypes.sizeof(nvq.RmsNormArgs), T=4, D=64, dtype=1, w_dtype=0, x=OK_PTR, weight=OK_PTR,
                        eps=1e-6, y=OK_PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return _lib().nvq_rms_norm(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(struct_size=8), EINVAL), (dict(dtype=2), EINVAL), (dict(w_dtype=-1), EINVAL), (dict(x=None), EINVAL),
    (dict(weight=None), EINVAL), (dict(y=None), EINVAL), (dict(residual=OK_PTR), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL), (dict(y8=OK_PTR), EINVAL),
    (dict(y=None, out_amax=OK_PTR, y8=OK_PTR, y8_scales=OK_PTR), EINVAL), (dict(group=16), EINVAL), (dict(group=-32), EINVAL),
    (dict(T=-1), ESHAPE), (dict(T=1 << 24), ESHAPE), (dict(D=0), ESHAPE), (dict(D=60), ESHAPE), (dict(D=32776), ESHAPE),
    (dict(x_ld=56), ESHAPE), (dict(y_ld=63), ESHAPE), (dict(h_ld=1), ESHAPE),
    (dict(D=96, y8=OK_PTR, y8_scales=OK_PTR, group=64), ESHAPE),
    (dict(x=OK_PTR + 8), EALIGN), (dict(x_ld=68), EALIGN), (dict(y=OK_PTR + 2), EALIGN), (dict(weight=OK_PTR + 4), EALIGN),
    (dict(y8=OK_PTR + 4, y8_scales=OK_PTR), EALIGN), (dict(rstd=OK_PTR + 2), EALIGN), (dict(out_amax=OK_PTR + 1), EALIGN),
    (dict(residual=OK_PTR, h=OK_PTR + 8), EALIGN), (dict(T=0, x=None, y=None), 0),
])
def test_norm(kw, rc):
    assert _norm(**kw) == rc


def _norm_grad(**kw):
    a = nvq.RmsNormGradArgs(struct_size=ctypes.sizeof(nvq.RmsNormGradArgs), T=4, D=64, dtype=1, w_dtype=0, dy=OK_PTR, h=OK_PTR,
                            weight=OK_PTR, rstd=OK_PTR, dx=OK_PTR, dweight=OK_PTR, ws=OK_PTR, ws_bytes=1 << 20)
    for k, v in kw.items():
        setattr(a, k, v)
    return _lib().nvq_rms_norm_backward(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(struct_size=0), EINVAL), (dict(dtype=5), EINVAL), (dict(dy=None), EINVAL), (dict(h=None), EINVAL),
    (dict(rstd=None), EINVAL), (dict(dx=None), EINVAL), (dict(weight=None), EINVAL), (dict(D=12), ESHAPE),
    (dict(D=40000), ESHAPE), (dict(T=1 << 30), ESHAPE), (dict(dh_ld=8), ESHAPE), (dict(dx=OK_PTR + 8), EALIGN),
    (dict(dh=OK_PTR + 4), EALIGN), (dict(dweight=OK_PTR + 2), EALIGN), (dict(dy_ld=66), EALIGN),
    (dict(ws=None), EWORKSPACE), (dict(ws_bytes=256), EWORKSPACE), (dict(ws=OK_PTR + 16), EALIGN),
    (dict(T=0, dy=None, h=None, rstd=None, dx=None, dweight=None, ws=None), 0),
])
def test_norm_gradient(kw, rc):
    assert _norm_grad(**kw) == rc


def _ce(backward=False, **kw):
    L = _lib()
    a = nvq.LinearCeArgs(struct_size=ctypes.sizeof(nvq.LinearCeArgs), T=4, D=64, V=100, x=OK_PTR, w=OK_PTR, targets=OK_PTR,
                         scale=1.0, loss=OK_PTR, lse=OK_PTR, dx=OK_PTR, dw=OK_PTR, dw_dtype=1, ws=OK_PTR, ws_bytes=1 << 40)
    for k, v in kw.items():
        setattr(a, k, v)
    return (L.nvq_linear_cross_entropy_backward if backward else L.nvq_linear_cross_entropy)(ctypes.byref(a), None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw,rc", [
    (dict(struct_size=16), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(targets=None), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(T=-1), ESHAPE), (dict(T=(1 << 23) + 1), ESHAPE),
    (dict(T=1 << 20, V=(1 << 19) + 1), ESHAPE), (dict(D=0), ESHAPE), (dict(D=63), ESHAPE), (dict(D=1 << 17), ESHAPE), (dict(V=0), ESHAPE), (dict(V=(1 << 24) + 1), ESHAPE),
    (dict(x_ld=56), ESHAPE), (dict(w_ld=8), ESHAPE), (dict(w_ld=(1 << 21) + 8), ESHAPE), (dict(x=OK_PTR + 8), EALIGN),
    (dict(w=OK_PTR + 2), EALIGN), (dict(w_ld=68), EALIGN), (dict(x_ld=71), EALIGN), (dict(targets=OK_PTR + 1), EALIGN),
    (dict(lse=OK_PTR + 2), EALIGN), (dict(ws=None), EWORKSPACE), (dict(ws_bytes=300), EWORKSPACE), (dict(ws=OK_PTR + 128), EALIGN),
])
def test_cross_entropy(backward, kw, rc):
    assert _ce(backward, **kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(dx=None, dw=None), EINVAL), (dict(lse=None), EINVAL), (dict(dw_dtype=3), EINVAL), (dict(dx_ld=32), ESHAPE),
    (dict(dw_ld=60), ESHAPE), (dict(dx=OK_PTR + 8), EALIGN), (dict(dw=OK_PTR + 4), EALIGN), (dict(dw_ld=68), EALIGN),
    (dict(dx_ld=66), EALIGN), (dict(dloss=OK_PTR + 3), EALIGN),
])
def test_cross_entropy_gradient(kw, rc):
    assert _ce(True, **kw) == rc


def test_cross_entropy_wants_an_output():
    assert _ce(loss=None, lse=None) == EINVAL


def test_workspaces_stay_far_below_the_logits():
    L = _lib()
    T, D, V = 65536, 4096, 131072
    assert L.nvq_linear_cross_entropy_workspace_bytes(T, D, V) < T * V * 4 // 60
    assert L.nvq_linear_cross_entropy_backward_workspace_bytes(T, D, V) < T * V * 2 // 4
    # refused sizes have the least workspace, not an overflow
    for bad in ((-1, 64, 10), (4, 7, 10), (4, 64, 0), (1 << 60, 64, 10)):
        assert L.nvq_linear_cross_entropy_workspace_bytes(*bad) == 256
        assert L.nvq_linear_cross_entropy_backward_workspace_bytes(*bad) == 256


def _list(items, count=None, **kw):
    n = len(items)
    a = nvq.TensorListArgs(ctypes.sizeof(nvq.TensorListArgs), n if count is None else count,
                           (ctypes.c_void_p * n)(*(i[0] for i in items)), (ctypes.c_int64 * n)(*(i[1] for i in items)),
                           (ctypes.c_int32 * n)(*(i[2] for i in items)))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("items,kw,rc", [
    ([(OK_PTR, 4, 0)], dict(struct_size=3), EINVAL), ([(OK_PTR, 4, 2)], {}, EINVAL), ([(None, 4, 0)], {}, EINVAL),
    ([(OK_PTR, -1, 0)], {}, ESHAPE), ([(OK_PTR, (1 << 42) + 1, 0)], {}, ESHAPE), ([(OK_PTR + 2, 4, 0)], {}, EALIGN),
    ([(OK_PTR + 1, 4, 1)], {}, EALIGN), ([(OK_PTR, 4, 0)], dict(count=-1), ESHAPE),
    ([(OK_PTR, 4, 0)], dict(count=(1 << 20) + 1), ESHAPE), ([(OK_PTR, 4, 0)], dict(data=None), EINVAL),
])
def test_tensor_lists(items, kw, rc):
    L = _lib()
    bad, good = _list(items, **kw), _list([(OK_PTR, 4, 0)])
    ws = ctypes.c_void_p(OK_PTR)
    assert L.nvq_grad_norm(ctypes.byref(bad), ws, ws, 1 << 20, None) == rc
    assert L.nvq_clip_grad_norm(ctypes.byref(bad), None, 1.0, ws, ws, 1 << 20, None) == rc
    assert L.nvq_clip_grad_norm(ctypes.byref(good), ctypes.byref(bad), 1.0, ws, ws, 1 << 20, None) == rc
    assert L.nvq_grad_norm_workspace_bytes(ctypes.byref(bad)) == 256


def test_clipping_refuses():
    L = _lib()
    one, two = _list([(OK_PTR, 4, 0)]), _list([(OK_PTR, 4, 0), (OK_PTR, 4, 0)])
    ws = ctypes.c_void_p(OK_PTR)

    def clip(out=None, max_norm=1.0, norm=ws, w=ws, size=1 << 20, grads=one):
        return L.nvq_clip_grad_norm(ctypes.byref(grads), None if out is None else ctypes.byref(out), max_norm, norm, w, size, None)

    assert clip(max_norm=-1.0) == EINVAL and clip(max_norm=float("nan")) == EINVAL and clip(norm=None) == EINVAL
    assert clip(norm=ctypes.c_void_p(OK_PTR + 2)) == EALIGN
    assert clip(out=two) == ESHAPE and clip(out=_list([(OK_PTR, 5, 0)])) == ESHAPE
    assert clip(out=_list([(OK_PTR, 4, 1)])) == EINVAL
    assert clip(w=None) == EWORKSPACE and clip(size=256) == EWORKSPACE and clip(w=ctypes.c_void_p(OK_PTR + 64)) == EALIGN
    assert L.nvq_grad_norm(None, ws, ws, 1 << 20, None) == EINVAL


@pytest.mark.parametrize("n", [3, 300])
def test_clipping_refuses_overlap(n):
    """Written tensors lie over no other of the call, neighbours and out_i over
    grads_i do not count (an element is 4 bytes); accepted calls stop at the
    workspace."""
    L = _lib()
    a, b = [(OK_PTR + 64 * i, 16, 0) for i in range(n)], [(OK_PTR + 64 * (n + i), 16, 0) for i in range(n)]
    ws = ctypes.c_void_p(OK_PTR)

    def clip(grads, out=None):
        out = None if out is None else ctypes.byref(_list(out))
        return L.nvq_clip_grad_norm(ctypes.byref(_list(grads)), out, 1.0, ws, None, 0, None)

    late = [(b[0][0] + 4, 16, 0)] + b[1:]
    inside = a[:2] + [(a[0][0] + 8, 16, 0)] + a[3:]
    for grads, out in ((a, None), (a, b), (a, a), (a[::-1], b), (a, b[::-1]), (a, a[:1] + b[1:]), (a[:1] * n, b), (inside, b),
                       (a[:1] + [(a[0][0], 0, 0)] + a[2:], None)):
        assert clip(grads, out) == EWORKSPACE
    for grads, out in ((a[:1] * n, None), (inside, None), (a, a[::-1]), (a, a[1:] + a[:1]), (a, b[:1] * n), (a, late),
                       (a, a[:1] + [(a[n - 1][0] + 4, 16, 0)] + b[2:]), (a, a[:1] + [(a[0][0] + 32, 16, 0)] + b[2:]),
                       (inside, inside)):
        assert clip(grads, out) == EINVAL


def test_binding_refuses_before_the_library():
    import torch

    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(100, 64, dtype=torch.bfloat16)
    y = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: nvq.nvq_rms_norm(x, w[0]), lambda: nvq.nvq_rms_norm_e4m3(x, w[0]),
                 lambda: nvq.nvq_rms_norm_backward(x, x, w[0], torch.zeros(4)),
                 lambda: nvq.nvq_linear_cross_entropy(x, w, y),
                 lambda: nvq.nvq_linear_cross_entropy_backward(x, w, y, torch.zeros(4)),
                 lambda: nvq.nvq_grad_norm([x]), lambda: nvq.nvq_clip_grad_norm([x], 1.0)):
        with pytest.raises(ValueError):
            call()


def test_norm_refuses_one_buffer_for_both_results():
    """y over h would leave the residual stream normalised."""
    other = OK_PTR + 0x10000
    assert _norm(residual=other, h=OK_PTR, y=OK_PTR) == EINVAL
    assert _norm(residual=OK_PTR, h=OK_PTR, y=OK_PTR) == EINVAL
    assert _norm(residual=OK_PTR, h=OK_PTR, y=OK_PTR, y8=other, y8_scales=other) == EINVAL
    # nothing is written: not a conflict
    assert _norm(T=0, residual=other, h=OK_PTR, y=OK_PTR) == 0


def test_clipping_allocates_nothing():
    """Where no memory is to be had a long list is judged as ever: accepted up to
    the workspace that is missing, or refused for its overlap."""
    import os
    import subprocess
    import sys

    _lib()
    program = """
import ctypes, resource, sys
import numpy as np
from qat_nvfp4_quantize_amd import nvq
L = nvq.load()
n = 1 << 18
size = np.full(n, 16, np.int64)
kind = np.zeros(n, np.int32)
order = np.random.default_rng(1).permutation(n)

def listed(at):
    return nvq.TensorListArgs(ctypes.sizeof(nvq.TensorListArgs), n, at.ctypes.data_as(ctypes.POINTER(ctypes.c_void_p)),
                              size.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), kind.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))

a = (0x100000 + 64 * order).astype(np.uint64)
b = a + np.uint64(64 * n)
late = b.copy()
late[n // 2] = a[n // 3] + np.uint64(60)
up, above = np.sort(a), np.sort(b)
tail = above.copy()
tail[0] -= np.uint64(4)
lists = [listed(v) for v in (a, b, late, up, above, tail)]
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (2 << 20),) * 2)
ws = ctypes.c_void_p(0x100000)
got = [L.nvq_clip_grad_norm(ctypes.byref(lists[i]), None if o is None else ctypes.byref(lists[o]), 1.0, ws, None, 0, None)
       for i, o in ((0, None), (0, 0), (0, 1), (0, 2), (3, None), (3, 3), (3, 4), (3, 5), (5, 3), (3, 0))]
sys.exit(0 if got == [-4, -4, -4, -1, -4, -4, -4, -1, -1, -1] else repr(got))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, cwd=root)
    assert r.returncode == 0, r.stderr[-500:]


def test_the_tiled_sizes_go_to_tiles():
    """The kernel for few tokens leaves a partial result (8 bytes a token) for each
    64 words, up to 512, tiles one for each 128: the workspace tells which it is."""
    from test_gpu_linear_ce import TILED, TILED_SIZES

    L = _lib()
    for T, D, V in [(T, 64, V) for T, V in TILED] + TILED_SIZES:
        tiles, few = (V + 127) // 128, min((V + 63) // 64, 512)
        assert 8 * T * tiles <= L.nvq_linear_cross_entropy_workspace_bytes(T, D, V) < 8 * T * few, (T, D, V)
    for T, D, V in [(40, 64, 5000), (300, 64, 1000)]:
        assert 8 * T * min((V + 63) // 64, 512) <= L.nvq_linear_cross_entropy_workspace_bytes(T, D, V)
