"""GPU parity of the paged NVFP4 cache's write and read back: bit-exact with
the oracle's quantizer and dequantizer at the cache's tensor scales, slots in
any order, padding, bad slots, strides, extreme scales, offsets past 32 bits."""
import numpy as np
import pytest

import oracle
from helpers import assert_bits_equal, log, to_np
from qat_nvfp4_quantize_amd import inputs

pytestmark = pytest.mark.gpu


def _nvq():
    from qat_nvfp4_quantize_amd import nvq

    return nvq


def _filled(nvq, P, H, S, D, ka=42.0, va=42.0):
    c = nvq.KvCache.empty(P, H, S, D, ka, va)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.fill_(0xA5)
    return c


def _expect(x, amax, dtype):
    """Oracle record and read-back values of rows [T, H, D] given as numpy."""
    T, H, D = x.shape
    codes, scales, st = oracle.quantize(np.ascontiguousarray(x.reshape(T * H, D)), amax_in=amax)
    deq = oracle.dequantize(codes, scales, st, out=dtype)
    return codes.reshape(T, H, D // 2), scales.reshape(T, H, D // 16), deq.reshape(T, H, D), st


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,H,D,S,amax", [(1, 1, 16, 16, 42.0), (67, 3, 128, 16, 42.0), (300, 2, 64, 64, 5.0),
                                          (41, 5, 256, 32, 42.0), (29, 2, 48, 128, 42.0), (9, 1, 512, 16, 3e38),
                                          (13, 2, 80, 16, 1e-36), (8, 1, 32, 16, 0.0)])
def test_append_and_gather_match_the_oracle(T, H, D, S, amax, dtype):
    import torch

    nvq = _nvq()
    log(f"[kvpages] T={T} H={H} D={D} S={S} amax={amax} {dtype}")
    r = np.random.default_rng(T + D)
    P = T // S + 3
    v_amax = 2 * amax if amax < 1e30 else amax
    c = _filled(nvq, P, H, S, D, amax, v_amax)
    size = min(amax, 1e30) / 4 if amax else 1.0
    fused = torch.from_numpy(r.standard_normal((T, 2 * H + 1, D)).astype(np.float32) * np.float32(size))
    fused[T // 2, 0] = 0.0
    fused[-1, :, 3] *= 50  # past the static amax
    fused = fused.to(getattr(torch, dtype)).cuda()
    k, v = fused[:, :H], fused[:, H + 1:]
    slots = r.permutation(P * S)[:T].astype(np.int32)
    if T > 5:
        slots[2] = -1
        slots[4] = -(2 ** 31)
    sl = torch.from_numpy(slots).cuda()
    ws = nvq.workspace(256, "cuda")
    nvq.nvq_kv_append(c, k, v, sl, ws=ws)
    assert nvq.device_status(ws) == 0
    live = slots >= 0
    pg, off = slots[live] // S, slots[live] % S
    touched = np.zeros((P, S), bool)
    touched[pg, off] = True
    for x, codes, scales, st in ((k, c.k_codes, c.k_scales, c.k_scale),
                                 (v, c.v_codes, c.v_scales.transpose(2, 3), c.v_scale)):
        # fp32 copies of bf16 rows: the oracle's decisions are those of the value
        oc, os_, _, ost = _expect(x.float().cpu().numpy(), amax if x is k else v_amax, "f32")
        assert float(st[0]) == ost
        assert_bits_equal(to_np(codes)[pg, :, off], oc[live], "codes")
        assert_bits_equal(to_np(scales)[pg, :, off], os_[live], "scales")
        assert (to_np(codes).transpose(0, 2, 1, 3)[~touched] == 0xA5).all()  # other slots keep their bytes
        assert (to_np(scales).transpose(0, 2, 1, 3)[~touched] == 0xA5).all()
    for out_dtype, name in ((torch.bfloat16, "bf16"), (torch.float32, "f32")):
        gk, gv = nvq.nvq_kv_gather(c, sl, out_dtype=out_dtype, ws=ws)
        assert nvq.device_status(ws) == 0
        for x, got, a in ((k, gk, amax), (v, gv, v_amax)):
            want = _expect(x.float().cpu().numpy(), a, name)[2].copy()
            want[~live] = 0
            assert_bits_equal(to_np(got), want, f"read back {name}")


def test_bad_slots_and_nonfinite_values_are_reported():
    import torch

    nvq = _nvq()
    c = _filled(nvq, 2, 2, 16, 32)
    k = torch.randn(4, 2, 32, device="cuda")
    ws = nvq.workspace(256, "cuda")
    before = [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    bad = torch.tensor([32, 2 ** 31 - 1, -1, 33], dtype=torch.int32, device="cuda")
    nvq.nvq_kv_append(c, k, k, bad, ws=ws)
    assert nvq.device_status(ws) == nvq.NVQ_STATUS_BAD_SLOT
    for t, b in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), before):
        assert torch.equal(t, b)
    gk, gv = nvq.nvq_kv_gather(c, bad, ws=ws)
    assert nvq.device_status(ws) == nvq.NVQ_STATUS_BAD_SLOT
    assert not gk.any() and not gv.any()
    good = torch.tensor([0, 5, 31, -1], dtype=torch.int32, device="cuda")
    nvq.nvq_kv_append(c, k, k, good, ws=ws)
    assert nvq.device_status(ws) == 0  # the word is cleared by each call
    k[1, 1, 7] = float("inf")
    nvq.nvq_kv_append(c, k, k, good, ws=ws)
    assert nvq.device_status(ws) == nvq.NVQ_STATUS_NONFINITE
    # the same slot read twice, and no token at all
    twice = torch.tensor([5, 5, 0], dtype=torch.int32, device="cuda")
    a, b = nvq.nvq_kv_gather(c, twice)
    assert torch.equal(a[0], a[1]) and torch.equal(b[0], b[1])
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    nvq.nvq_kv_append(c, k[:0], k[:0], none)
    assert nvq.nvq_kv_gather(c, none)[0].shape == (0, 2, 32)


def test_two_tokens_in_one_slot_leave_bytes_of_theirs():
    import torch

    nvq = _nvq()
    c = _filled(nvq, 1, 1, 16, 64)
    k = torch.randn(2, 1, 64, device="cuda")
    one = []
    for i in range(2):
        nvq.nvq_kv_append(c, k[i:i + 1], k[i:i + 1], torch.tensor([3], dtype=torch.int32, device="cuda"))
        one.append((c.k_codes[0, 0, 3].clone(), c.v_scales[0, 0, :, 3].clone()))
    nvq.nvq_kv_append(c, k, k, torch.tensor([3, 3], dtype=torch.int32, device="cuda"))
    got = c.k_codes[0, 0, 3], c.v_scales[0, 0, :, 3]
    for x, a, b in zip(got, *one):
        assert ((x == a) | (x == b)).all()


def test_slots_past_32_bits_of_bytes():
    import torch

    nvq = _nvq()
    H, S, D = 8, 64, 128
    P = (2 ** 32) // (H * S * D // 2) + 40  # the last pages lie past 4 GiB of codes
    c = nvq.KvCache.empty(P, H, S, D, 42.0, 42.0)
    k = torch.randn(50, H, D, device="cuda").to(torch.bfloat16)
    v = torch.randn(50, H, D, device="cuda").to(torch.bfloat16)
    slots = (P * S - 1 - 3 * torch.arange(50, dtype=torch.int32, device="cuda")).to(torch.int32)
    nvq.nvq_kv_append(c, k, v, slots)
    small = _filled(nvq, 4, H, S, D)
    low = torch.arange(50, dtype=torch.int32, device="cuda")
    nvq.nvq_kv_append(small, k, v, low)
    for a, b in zip(nvq.nvq_kv_gather(c, slots), nvq.nvq_kv_gather(small, low)):
        assert torch.equal(a, b)


def test_append_equals_the_quantizer_of_dense_rows():
    """The bytes are those of nvfp4_quantize with the cache's static amax."""
    import torch

    nvq = _nvq()
    new = inputs.kv_append()
    T, D = new.shape[1], new.shape[2]
    x = torch.from_numpy(new.view(np.int16)).view(torch.bfloat16).cuda()
    amax = torch.full((2,), inputs.KV_STATIC_AMAX, dtype=torch.float32, device="cuda")
    codes, scales, st, _, _ = nvq.nvfp4_quantize(x, amax_in=amax)
    c = _filled(nvq, T // 64 + 1, 1, 64, D, inputs.KV_STATIC_AMAX, inputs.KV_STATIC_AMAX)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    nvq.nvq_kv_append(c, x[0][:, None], x[1][:, None], slots)
    assert torch.equal(c.k_codes[:, 0].reshape(-1, D // 2)[:T], codes[0])
    assert torch.equal(c.k_scales[:, 0].reshape(-1, D // 16)[:T], scales[0])
    assert torch.equal(c.v_codes[:, 0].reshape(-1, D // 2)[:T], codes[1])
    assert torch.equal(c.v_scales[:, 0].transpose(1, 2).reshape(-1, D // 16)[:T], scales[1])
    assert float(c.k_scale[0]) == float(st[0]) and float(c.v_scale[0]) == float(st[1])


def test_either_output_may_be_left_out():
    import ctypes

    import torch

    nvq = _nvq()
    T, H, D, S = 33, 3, 64, 16
    cache = _filled(nvq, 6, H, S, D)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(T, H, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    slots = torch.randperm(6 * S, generator=g)[:T].to(torch.int32).cuda()
    nvq.nvq_kv_append(cache, k, v, slots)
    want = nvq.nvq_kv_gather(cache, slots)
    for i in range(2):
        got = torch.full((T, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
        dst = [None, None]
        dst[i] = got.data_ptr()
        rc = nvq.load().nvq_kv_gather(ctypes.byref(cache.args), slots.data_ptr(), T, *dst, nvq._dtype_code(got), None,
                                      0, torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and torch.equal(got, want[i])
