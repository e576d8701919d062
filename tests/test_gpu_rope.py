"""GPU parity of the rotary positions with a 64-bit evaluation: both pair
layouts, parts of the head, far positions, the gradient, strided and in-place
rows, sizes off the vector path."""
import numpy as np
import pytest

import attention_reference as ref
from helpers import log

pytestmark = pytest.mark.gpu


def _nvq():
    from qat_nvfp4_quantize_amd import nvq

    return nvq


def _check(y, x, pos, f, inter, mag, inverse, what):
    import torch

    want, bound = ref.rope(x.detach().float().cpu().numpy(), pos.cpu().numpy(), f.cpu().numpy(), inter, mag, inverse)
    if x.dtype == torch.bfloat16:
        bound = bound + ref.BF16 * np.abs(want)
    off = np.abs(y.float().cpu().numpy().astype(np.float64) - want)
    assert (off <= bound).all(), (what, float((off - bound).max()))
    rot = 2 * len(f)
    assert torch.equal(y[..., rot:].cpu(), x[..., rot:].cpu()), what  # the rest is copied


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 2, 2), (3, 5, 128, 128), (130, 7, 64, 32), (17, 3, 80, 20),
                                       (33, 2, 256, 256), (5, 1, 1000, 998), (2, 3, 4096, 4096), (70, 40, 128, 64)])
def test_rope_matches_64_bits(T, H, D, rot, inter, dtype):
    import torch

    nvq = _nvq()
    log(f"[rope] T={T} H={H} D={D} rot={rot} inter={inter} {dtype}")
    g = torch.Generator().manual_seed(T * D + rot)
    x = (torch.randn(T, H, D, generator=g) * 3).to(getattr(torch, dtype)).cuda()
    pos = torch.randint(-(2 ** 31), 2 ** 31 - 1, (T,), generator=g, dtype=torch.int64).to(torch.int32).cuda()
    pos[0] = 2 ** 31 - 1
    pos[T // 2] = 0
    f, m = nvq.nvq_rope_frequencies(rot, kind=nvq.NVQ_ROPE_RAMP, factor=16.0, orig_len=4096.0)
    f = f.cuda()
    for inverse in (False, True):
        y = nvq.nvq_rope(x, pos, f, interleaved=inter, magnitude=m, inverse=inverse)
        # the library's angle at position 2^31 is off by 2^-20 at most
        want, bound = ref.rope(x.float().cpu().numpy(), pos.cpu().numpy(), f.cpu().numpy(), inter, m, inverse)
        u = np.abs(x.float().cpu().numpy().astype(np.float64))
        bound = bound + 2.0 ** -20 * m * 2 * u.max() + (ref.BF16 * np.abs(want) if dtype == "bfloat16" else 0)
        off = np.abs(y.float().cpu().numpy() - want)
        assert (off <= bound).all(), float((off - bound).max())
        near = (pos % 100000).to(torch.int32)
        _check(nvq.nvq_rope(x, near, f, interleaved=inter, magnitude=m, inverse=inverse), x, near, f, inter, m,
               inverse, "near positions")


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("pad,rot", [(8, 64), (3, 64), (0, 24)])
def test_rope_strided_in_place_and_gradient(inter, pad, rot):
    import torch

    nvq = _nvq()
    g = torch.Generator().manual_seed(pad + rot)
    T, H, D = 37, 6, 64
    fused = torch.randn(T, H + 2, D + pad, generator=g).to(torch.bfloat16).cuda()
    x = fused[:, 1:H + 1, :D]
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 911
    f = nvq.nvq_rope_frequencies(rot)[0].cuda()
    y = nvq.nvq_rope(x, pos, f, interleaved=inter)
    _check(y, x, pos, f, inter, 1.0, False, "strided")
    before = fused.clone()
    nvq.nvq_rope(x, pos, f, interleaved=inter, out=x)
    assert torch.equal(x, y)
    keep = torch.ones_like(fused, dtype=torch.bool)
    keep[:, 1:H + 1, :D] = False
    assert torch.equal(fused[keep], before[keep])  # nothing beside the rows is written
    # heads-first memory
    z = torch.randn(H, T, D, generator=g).cuda().transpose(0, 1)
    out = torch.empty(H, T, D, device="cuda").transpose(0, 1)
    assert nvq.nvq_rope(z, pos, f, interleaved=inter, out=out) is out
    _check(out, z, pos, f, inter, 1.0, False, "heads first")
    # <g, J dx> = <J^T g, dx> in 64 bits: the inverse call is the gradient (fp32 in and out)
    gy, dx = (torch.randn(T, H, D, generator=g).cuda() for _ in range(2))
    fwd = nvq.nvq_rope(dx, pos, f, interleaved=inter, magnitude=1.25)
    bwd = nvq.nvq_rope(gy, pos, f, interleaved=inter, magnitude=1.25, inverse=True)
    a, b = (fwd.double() * gy.double()).sum(), (bwd.double() * dx.double()).sum()
    # each element of a call is off by 8 U32 m (|a| + |b|) at most, so each product by that of its pair
    def pair(x):
        x, h = x[..., :rot].double().abs(), rot // 2
        return x[..., 0::2] + x[..., 1::2] if inter else x[..., :h] + x[..., h:]

    assert abs(float(a - b)) <= 2 * 8 * ref.U32 * 1.25 * float((pair(gy) * pair(dx)).sum())
    # against a difference of the forward call, which is linear: J (x + d) - J x = J d
    x32 = torch.randn(T, H, D, generator=g).cuda()
    diff = nvq.nvq_rope(x32 + dx, pos, f, interleaved=inter).double() - nvq.nvq_rope(x32, pos, f, interleaved=inter).double()
    jd = nvq.nvq_rope(dx, pos, f, interleaved=inter).double()
    room = 16 * ref.U32 * 2 * (x32.abs().max() + dx.abs().max()).item() * 2
    assert float((diff - jd).abs().max()) <= room


def test_rope_of_nothing_and_special_values():
    import torch

    nvq = _nvq()
    f = nvq.nvq_rope_frequencies(32)[0].cuda()
    empty = torch.empty(0, 4, 64, device="cuda")
    assert nvq.nvq_rope(empty, torch.empty(0, dtype=torch.int32, device="cuda"), f).shape == (0, 4, 64)
    x = torch.ones(2, 1, 64, device="cuda", dtype=torch.bfloat16)
    x[0, 0, 3] = float("inf")
    x[1, 0, 40] = float("nan")  # past the rotated part
    y = nvq.nvq_rope(x, torch.tensor([1, 2], dtype=torch.int32, device="cuda"), f).float().cpu()
    assert not torch.isfinite(y[0, 0, [3, 19]]).any()
    ok = torch.ones(2, 64, dtype=torch.bool)
    ok[0, [3, 19]] = False
    ok[1, 40] = False
    assert torch.isfinite(y[:, 0][ok]).all() and torch.isnan(y[1, 0, 40])
