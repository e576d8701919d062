"""Host-side refusals of the rotary, paged-cache and attention entry points
(nothing is launched, so they run without a GPU), the rotation's frequencies,
and the tests' own plain forms against closed cases."""
import ctypes
import math
import os

import numpy as np
import pytest

import attention_reference as ref
from qat_nvfp4_quantize_amd import nvq

P = ctypes.c_void_p
FAKE = P(0x1000)  # never dereferenced: every call below fails validation first


def _lib():
    if not os.path.exists(nvq.LIB_PATH):
        pytest.skip("libnvq.so not built")
    return nvq.load()


def _cache(**over):
    c = nvq.KvCacheArgs(ctypes.sizeof(nvq.KvCacheArgs), 0x1000, 0x1000, 0x1000, 0x1000, 0x1000, 0x1000, 8, 16, 2, 128)
    for k, v in over.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def test_rope_refusals():
    L = _lib()

    def call(x=FAKE, dtype=1, T=4, H=2, D=64, xt=0, xh=0, pos=FAKE, f=FAKE, rot=64, layout=0, y=P(0x9000), yt=0, yh=0):
        return L.nvq_rope(x, dtype, T, H, D, xt, xh, pos, f, rot, layout, 1.0, 0, y, yt, yh, None)

    assert call(dtype=2) == -1 and call(layout=2) == -1
    for bad in (dict(rot=0), dict(rot=3), dict(rot=66), dict(D=1, rot=2), dict(D=8192), dict(T=-1), dict(H=65536),
                dict(T=1 << 24), dict(xt=-1), dict(yh=63), dict(yt=63), dict(yt=64, yh=64), dict(yt=64, yh=255)):
        assert call(**bad) == -2, bad
    for bad in (dict(x=None), dict(y=None), dict(pos=None), dict(f=None), dict(y=FAKE, xt=256)):
        assert call(**bad) == -1, bad
    for bad in (dict(x=P(0x1001)), dict(dtype=0, y=P(0x9002)), dict(pos=P(0x1002)), dict(f=P(0x1004))):
        assert call(**bad) == -3, bad
    assert call(T=0, x=None, y=None, pos=None, f=None) == 0 and call(H=0, x=None) == 0


def test_rope_frequencies():
    _lib()
    f, m = nvq.nvq_rope_frequencies(64, base=500.0)
    want = 500.0 ** (-np.arange(32) / 32)
    np.testing.assert_allclose(f.numpy(), want, rtol=1e-14)
    assert m == 1.0
    np.testing.assert_allclose(nvq.nvq_rope_frequencies(64, 500.0, nvq.NVQ_ROPE_LINEAR, 8.0)[0].numpy(), want / 8,
                               rtol=1e-14)
    b = nvq.nvq_rope_frequencies(64, 500.0, nvq.NVQ_ROPE_BASE, 8.0)[0].numpy()
    assert b[0] == 1.0 and abs(b[-1] / (want[-1] / 8) - 1) < 1e-13  # fastest kept, slowest divided
    r, m = nvq.nvq_rope_frequencies(64, 500.0, nvq.NVQ_ROPE_RAMP, 8.0, orig_len=2048.0, slow=1.0, fast=32.0)
    turns = 2048 * want / (2 * math.pi)
    part = np.clip((turns - 1) / 31, 0, 1)
    np.testing.assert_allclose(r.numpy(), want * part + want / 8 * (1 - part), rtol=1e-14)
    assert abs(m - (0.1 * math.log(8) + 1)) < 1e-7
    assert (r.numpy()[turns >= 32] == want[turns >= 32]).all() and (turns < 1).any()
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=2, kind=2), dict(rot_dim=8, kind=4),
                dict(rot_dim=8, base=0.0), dict(rot_dim=8, base=float("nan")), dict(rot_dim=8, kind=1, factor=0.5),
                dict(rot_dim=8, kind=2, base=1.0), dict(rot_dim=8, kind=3, factor=2.0),
                dict(rot_dim=8, kind=3, factor=2.0, orig_len=10.0, slow=4.0, fast=4.0)):
        with pytest.raises(nvq.NvqError):
            nvq.nvq_rope_frequencies(**bad)


def test_cache_refusals():
    L = _lib()

    def append(c=None, k=FAKE, v=FAKE, dtype=1, T=4, ld=(0, 0, 0, 0), slots=FAKE, ws=None, n=0):
        return L.nvq_kv_append(c or _cache(), k, v, dtype, T, *ld, slots, ws, n, None)

    def gather(c=None, slots=FAKE, T=4, k=FAKE, v=FAKE, dtype=1, ws=None, n=0):
        return L.nvq_kv_gather(c or _cache(), slots, T, k, v, dtype, ws, n, None)

    for call in (append, gather):
        for bad in (dict(struct_size=8), dict(k_codes=None), dict(v_scales=None), dict(k_tensor_scale=None)):
            assert call(c=_cache(**bad)) == -1, bad
        for bad in (dict(page_size=8), dict(page_size=24), dict(page_size=131072), dict(head_dim=24),
                    dict(head_dim=528), dict(head_dim=0), dict(heads=0), dict(heads=65536), dict(num_pages=0),
                    dict(num_pages=2 ** 27)):
            assert call(c=_cache(**bad)) == -2, bad
        for bad in (dict(k_codes=0x1008), dict(v_scales=0x1004), dict(v_tensor_scale=0x1002)):
            assert call(c=_cache(**bad)) == -3, bad
        assert call(dtype=3) == -1 and call(T=-1) == -2 and call(T=1 << 24) == -2 and call(slots=None) == -1
        assert call(slots=P(0x1002)) == -3 and call(k=P(0x1008)) == -3
        assert call(ws=P(0x1010), n=256) == -3 and call(ws=FAKE, n=255) == -4
        assert call(T=0, k=None, v=None, slots=None) == 0
    assert L.nvq_kv_append(None, FAKE, FAKE, 1, 4, 0, 0, 0, 0, FAKE, None, 0, None) == -1
    assert append(k=None) == -1 and append(v=None) == -1
    assert append(ld=(252, 0, 0, 0)) == -3 and append(dtype=0, ld=(0, 0, 0, 130)) == -3
    assert append(ld=(-256, 0, 0, 0)) == -2
    assert gather(k=None, v=None) == -1


def _args(**over):
    a = nvq.PagedAttentionArgs()
    a.struct_size = ctypes.sizeof(a)
    a.total_q, a.B, a.q_heads, a.causal, a.softmax_scale = 4, 2, 8, 1, 0.1
    for f in ("q", "cu_q", "kv_len", "block_table", "out", "ws"):
        setattr(a, f, 0x1000)
    a.table_width, a.ws_bytes = 4, 1 << 40
    for k, v in over.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def test_attention_refusals():
    L = _lib()

    def call(c=None, **over):
        return L.nvq_paged_attention(c or _cache(), _args(**over), None)

    assert L.nvq_paged_attention(None, _args(), None) == -1 and L.nvq_paged_attention(_cache(), None, None) == -1
    for bad in (dict(struct_size=8), dict(causal=2), dict(window=-1), dict(causal=0, window=5),
                dict(softmax_scale=float("inf")), dict(softmax_scale=float("nan")), dict(q=None), dict(out=None),
                dict(cu_q=None), dict(kv_len=None), dict(block_table=None), dict(ws=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(total_q=-1), dict(total_q=1 << 24), dict(B=-1), dict(B=65536), dict(max_q=-1), dict(q_heads=7),
                dict(q_heads=0), dict(q_heads=65536), dict(table_width=-1), dict(table_width=2 ** 27), dict(table_ld=3),
                dict(q_ld_t=-8), dict(out_ld_h=64), dict(out_ld_t=64), dict(out_ld_t=128, out_ld_h=128)):
        assert call(**bad) == -2, bad
    for bad in (dict(q=0x1008), dict(out=0x1002), dict(q_ld_t=1028), dict(q_ld_h=132), dict(out_ld_t=1028),
                dict(cu_q=0x1002), dict(lse=0x1001), dict(ws=0x1010)):
        assert call(**bad) == -3, bad
    # products of sizes: rows and heads, sequences and heads, table entries, 128-key units
    for bad, c in ((dict(total_q=1 << 20, q_heads=1032), None),
                   (dict(B=32769, q_heads=64, table_width=1), dict(heads=64)),
                   (dict(B=65535, table_width=16385), None),
                   (dict(B=64, table_width=2 ** 16 - 1), dict(page_size=65536))):
        assert call(c=_cache(**c) if c else None, **bad) == -2, bad
    assert call(softmax_scale=3e38) == -1  # not finite in base 2
    assert call(ws_bytes=255) == -4
    assert call(c=_cache(page_size=8)) == -2 and call(c=_cache(head_dim=520)) == -2 and call(c=_cache(heads=3)) == -2
    assert call(c=_cache(k_scales=0x1008)) == -3
    # the workspace query needs sizes only, and one workspace smaller is refused
    for over in (dict(), dict(total_q=4096, max_q=2048), dict(total_q=64, B=64, max_q=1, table_width=4096)):
        n = L.nvq_paged_attention_workspace_bytes(_cache(k_codes=None), _args(q=None, ws=None, **over))
        assert n >= 256 and call(ws_bytes=n - 1, **over) == -4


def test_binding_refuses_tensors_off_the_gpu():
    import torch

    x = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError):
        nvq.nvq_rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
    u = torch.zeros(2, 2, 16, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        nvq.KvCache(u, u, u, u, torch.ones(1), torch.ones(1))


def test_plain_forms_in_closed_cases():
    # a quarter turn of the only pair; both layouts agree on one pair
    x = np.array([[[3.0, 4.0, 9.0]]])
    for inter in (False, True):
        y, _ = ref.rope(x, np.array([1]), [math.pi / 2], inter, 2.0, False)
        np.testing.assert_allclose(y, [[[-8.0, 6.0, 9.0]]], atol=1e-14)
        y, _ = ref.rope(x, np.array([1]), [math.pi / 2], inter, 1.0, True)
        np.testing.assert_allclose(y, [[[4.0, -3.0, 9.0]]], atol=1e-14)
    # interleaved and half layouts are the same rotation of permuted elements
    r = np.random.default_rng(0)
    z, pos, f = r.standard_normal((5, 2, 8)), np.arange(5), 0.3 ** np.arange(4)
    order = [0, 2, 4, 6, 1, 3, 5, 7]
    np.testing.assert_allclose(ref.rope(z, pos, f, True, 1, False)[0][..., order],
                               ref.rope(z[..., order], pos, f, False, 1, False)[0], atol=1e-14)
    # values: codes 7 (6.0) and 9 (-0.5) with scale 0x38 (1.0), and a subnormal scale 2^-9
    v = ref.stored_values(np.full((1, 8), 0x97, np.uint8), np.array([[0x38]], np.uint8), 0.5)
    assert (v[0, 0::2] == 3.0).all() and (v[0, 1::2] == -0.25).all()
    assert ref.stored_values(np.full((1, 8), 0x22, np.uint8), np.array([[1]], np.uint8), 1.0)[0, 0] == 2.0 ** -9
    # equal scores average the visible values; window and causal limits; an empty row
    k = np.zeros((4, 1, 2))
    val = np.arange(8.0).reshape(4, 1, 2)
    q = np.ones((3, 2, 2))
    out, lse, _ = ref.attention(q, k, val, 1, 1.0, True, 0)
    np.testing.assert_allclose(out[:, 0, 0], [1.0, 2.0, 3.0])
    np.testing.assert_allclose(lse[:, 0], np.log([2.0, 3.0, 4.0]))
    out, _, _ = ref.attention(q, k, val, 1, 1.0, True, 2)
    np.testing.assert_allclose(out[:, 0, 0], [1.0, 3.0, 5.0])
    out, lse, _ = ref.attention(q, k, val, -2, 1.0, True, 0)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and out[2, 0, 1] == 1.0
