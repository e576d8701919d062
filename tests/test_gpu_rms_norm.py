"""The RMS norm with the residual's addition, its 8-bit output and its gradient
against 64-bit forms."""
import pytest

import trainer_reference as ref
from helpers import log

pytestmark = pytest.mark.gpu


def _nvq():
    from qat_nvfp4_quantize_amd import nvq

    return nvq


def _inputs(T, D, dtype, wdtype, seed=0, big=1.0):
    import torch

    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + D)
    x, res, dy, dh = (torch.randn(T, D, generator=g) * big for _ in range(4))
    x[:, 3 % D] *= 30
    w = 1 + 0.2 * torch.randn(D, generator=g)
    t = getattr(torch, dtype)
    return [v.to(t).cuda() for v in (x, res, dy, dh)] + [w.to(getattr(torch, wdtype)).cuda()]


SIZES = [(1, 8), (2, 64), (3, 136), (7, 512), (5, 1000), (33, 1024), (64, 2048), (9, 2056), (4, 4096), (3, 5000), (2, 7168),
         (3, 8200), (2, 16384), (2, 32768), (700, 96), (1500, 256), (2, 24), (18, 128), (4500, 128), (35, 264),
         (9, 520), (5, 8192), (3, 16392), (300, 9000)]


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("dtype,wdtype", [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "float32"),
                                          ("float32", "bfloat16")])
def test_norm_and_gradient_match_64_bits(T, D, dtype, wdtype):
    import torch

    nvq = _nvq()
    log(f"[norm] T={T} D={D} {dtype} {wdtype}")
    x, res, dy, dh, w = _inputs(T, D, dtype, wdtype)
    e = ref.round_error(x.dtype)
    for residual in (None, res):
        (y, h, r), (e_y, e_r) = ref.rms_norm(x, residual, w, 1e-6)
        amax = torch.full((1,), 7e30, device="cuda")
        got_y, got_h, got_r = nvq.nvq_rms_norm(x, w, 1e-6, residual=residual, want_rstd=True, out_amax=amax)
        assert torch.equal(got_h, h) and (residual is not None or got_h is x)
        ref.within(got_r, r, e_r, "rstd")
        ref.within(got_y, y, e_y + e * (y.abs() + e_y), "y")
        assert float(amax) == float(got_y.abs().max())
        (dx, dw), (e_dx, e_dw) = ref.rms_norm_grad(dy, h, w, got_r, dh)
        got_dx, got_dw = nvq.nvq_rms_norm_backward(dy, got_h, w, got_r, dh=dh)
        ref.within(got_dx, dx, e_dx, "dx")
        ref.within(got_dw, dw, e_dw, "dweight")
        (dx, dw), (e_dx, _) = ref.rms_norm_grad(dy, h, w, got_r, None)
        again = got_dw.clone()
        got_dx, acc = nvq.nvq_rms_norm_backward(dy, got_h, w, got_r, dw=again, accumulate=True)
        ref.within(got_dx, dx, e_dx, "dx without dh")
        assert acc is again
        ref.within(acc, 2 * dw, 2 * e_dw + 2 * ref.U32 * 2 * dw.abs(), "dweight twice")
        only, none = nvq.nvq_rms_norm_backward(dy, got_h, w, got_r, want_dw=False)
        assert none is None and torch.equal(only, got_dx)


@pytest.mark.parametrize("T,D,group", [(1, 128, 128), (5, 96, 32), (3, 1024, 128), (64, 4096, 128), (2, 7168, 128), (9, 448, 64),
                                       (4, 32768, 128), (3, 1000, 0), (1, 8, 0), (130, 4096, 0), (2, 16384, 0), (300, 640, 128),
                                       (37, 128, 64), (50, 256, 32), (19, 256, 0), (21, 512, 128), (70, 24, 0), (3, 12288, 64)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_eight_bit_output(T, D, group, dtype):
    import torch

    nvq = _nvq()
    log(f"[norm e4m3] T={T} D={D} group={group} {dtype}")
    x, res, _, _, w = _inputs(T, D, dtype, "float32", seed=5)
    (y, h, r), (e_y, e_r) = ref.rms_norm(x, res, w, 1e-5)
    codes, scales, got_h, rstd = nvq.nvq_rms_norm_e4m3(x, w, 1e-5, residual=res, group=group, want_rstd=True)
    assert torch.equal(got_h, h)
    ref.within(rstd, r, e_r, "rstd")
    n = group or D
    top = y.reshape(T, D // n, n).abs().amax(-1)
    e_top = e_y.reshape(T, D // n, n).amax(-1)
    ref.within(scales, top / 448, (e_top + 2 * ref.U32 * top) / 448, "scales")
    s = scales.double().repeat_interleave(n, 1)
    # half a step of E4M3 (relative, or of its 2^-9 grid below 2^-6), and the rounding of scale and y
    room = s * torch.maximum(ref.E4M3 * (y / s).abs(), torch.full_like(y, 2.0 ** -10)) + (e_y + 2 * ref.U32 * y.abs()) * (1 + ref.E4M3)
    ref.within(codes.float().double() * s, y, room, "values")
    big = codes.float().abs().reshape(T, D // n, n).amax(-1)
    assert bool((big == 448).all())  # every group uses the whole range
    # the codes themselves: those of the quotients of exact products (48 bits in fp64), ties to even
    prod = h.double() * w.double()
    part = prod.reshape(T, D // n, n)
    q = 448 * part / part.abs().amax(-1, keepdim=True)
    assert torch.equal(codes.float().double(), ref.nearest_e4m3(q).reshape(T, D))


@pytest.mark.parametrize("group", [128, 32, 0])
def test_eight_bit_ties(group):
    """bf16 rows and weights of few bits: many quotients are exact midpoints."""
    import torch

    nvq = _nvq()
    g = torch.Generator().manual_seed(11)
    T, D = 40, 1024
    x = (torch.randint(-28, 29, (T, D), generator=g) / 4).to(torch.bfloat16).cuda()
    x[:, ::32] = 7.0
    w = (torch.randint(1, 3, (D,), generator=g) / 2).to(torch.bfloat16).cuda()
    codes, _, _, _ = nvq.nvq_rms_norm_e4m3(x, w, group=group)
    n = group or D
    part = (x.double() * w.double()).reshape(T, D // n, n)
    q = 448 * part / part.abs().amax(-1, keepdim=True)
    want = ref.nearest_e4m3(q)
    tied = ref.nearest_e4m3(q * (1 + 2.0 ** -40)) != ref.nearest_e4m3(q * (1 - 2.0 ** -40))
    assert int(tied.sum()) > 1000
    assert torch.equal(codes.float().double(), want.reshape(T, D))


def test_rows_of_zeros_nan_and_extreme_size():
    import torch

    nvq = _nvq()
    D = 256
    w = torch.ones(D, device="cuda")
    x = torch.zeros(6, D, device="cuda")
    x[1] = 1e30      # squares beyond fp32
    x[2] = 1e-30     # squares below it
    x[3, 7] = float("nan")
    x[4, 200] = float("inf")
    x[5] = torch.linspace(-3, 3, D)
    y, h, r = nvq.nvq_rms_norm(x, w, 0.0, want_rstd=True)
    assert h is x and bool(y[0].isnan().all())  # 0 * (1 / 0), as the formula has it
    ref.within(y[1], torch.ones(D, device="cuda").double(), 8 * ref.U32 * torch.ones(D, device="cuda").double(), "large")
    ref.within(y[2], torch.ones(D, device="cuda").double(), 8 * ref.U32 * torch.ones(D, device="cuda").double(), "small")
    assert bool(y[3].isnan().all()) and bool(y[4, 200].isnan()) and bool((y[4, :200] == 0).all())
    y, _, r = nvq.nvq_rms_norm(x, w, 1e-6, want_rstd=True)
    assert bool((y[0] == 0).all()) and float(r[0]) == 1000.0
    codes, scales, _, _ = nvq.nvq_rms_norm_e4m3(x, w, 1e-6, group=128)
    c = codes.float()
    assert bool((c[0] == 0).all()) and float(scales[0, 0]) == 2.0 ** -126
    assert bool(c[3].isnan().all()) and bool(scales[3].isnan().all())
    assert bool((c[4, :128] == 0).all()) and bool(c[4, 128:].isnan().all()) and bool(scales[4, 1].isnan())
    # large rows, ties (1 + 2^-4 of the grid's 1 and 9/8) to the even code, the signs of zeros
    w2 = torch.ones(128, device="cuda")
    t = torch.full((1, 128), 448.0, device="cuda")
    t[0, 1:8] = torch.tensor([1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, -(2.0 ** -11), 17.0])
    codes, scales, _, _ = nvq.nvq_rms_norm_e4m3(t * 2.0 ** 60, w2, 0.0, group=128)
    want = torch.tensor([448, 1.0, 1.25, -1.0, 0.0, 2.0 ** -8, -0.0, 16.0], device="cuda")
    assert torch.equal(codes[0, :8].float(), want) and bool(torch.signbit(codes[0, 6].float()))
    assert float(c[5].abs().max()) == 448
    # bf16 numbers below the normal ones keep their bits through the addition
    tiny = (torch.arange(-128, 128, device="cuda", dtype=torch.int16) << 0).view(torch.bfloat16).reshape(1, 256)
    tiny = torch.where(tiny.isnan(), 0.0, tiny.float()).to(torch.bfloat16)
    _, h, _ = nvq.nvq_rms_norm(tiny, w, 1e-6, residual=torch.zeros_like(tiny))
    assert torch.equal(h.view(torch.int16) & 0x7FFF, tiny.view(torch.int16) & 0x7FFF)
    # a NaN reaches the row's amax word too
    amax = torch.zeros(1, device="cuda")
    nvq.nvq_rms_norm(x, w, 1e-6, out_amax=amax)
    assert bool(amax.isnan().all())


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_strided_and_in_place(dtype):
    import torch

    nvq = _nvq()
    T, D = 37, 264
    x, res, dy, dh, w = _inputs(T, D, dtype, "float32", seed=9)
    y, h, r = nvq.nvq_rms_norm(x, w, residual=res, want_rstd=True)
    dx, dw = nvq.nvq_rms_norm_backward(dy, h, w, r, dh=dh)

    def wide(t, left):
        b = torch.full((T, D + 40), 99.0, dtype=t.dtype, device="cuda")
        b[:, left:left + D] = t
        return b, b[:, left:left + D]

    (bx, xs), (br, rs), (by, ys), (bh, hs) = wide(x, 8), wide(res, 16), wide(x, 24), wide(x, 32)
    y2, h2, r2 = nvq.nvq_rms_norm(xs, w, residual=rs, want_rstd=True, out=ys, residual_out=hs)
    assert y2 is ys and h2 is hs
    assert torch.equal(ys, y) and torch.equal(hs, h) and torch.equal(r2, r)
    assert bool((by[:, :24] == 99).all()) and bool((by[:, 24 + D:] == 99).all()) and bool((bh[:, :32] == 99).all())
    (bd, ds), (bg, gs), (bo, os_) = wide(dy, 8), wide(dh, 8), wide(dy, 16)
    dx2, dw2 = nvq.nvq_rms_norm_backward(ds, hs, w, r, dh=gs, out=os_)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and bool((bo[:, 16 + D:] == 99).all())
    # in place: y over x, h over the residual, dx over dh
    xi, ri, gi = x.clone(), res.clone(), dh.clone()
    y3, h3, _ = nvq.nvq_rms_norm(xi, w, residual=ri, out=xi, residual_out=ri)
    assert y3 is xi and h3 is ri and torch.equal(xi, y) and torch.equal(ri, h)
    dx3, _ = nvq.nvq_rms_norm_backward(dy, h, w, r, dh=gi, out=gi)
    assert torch.equal(dx3, dx)
    for over in (dy.clone(), h.clone()):
        a, b = (over, h) if torch.equal(over, dy) else (dy, over)
        got, got_dw = nvq.nvq_rms_norm_backward(a, b, w, r, dh=dh, out=over)
        assert torch.equal(got, dx) and torch.equal(got_dw, dw)


def test_gradient_against_differences_of_the_norm():
    """fp32: y at x + u and x - u.  The central difference is off by a third of
    the third derivative; with steps of 2^-10 of a row of size 1 that is below
    2^-24 of |y|, under the rounding of y, which is what the bound counts."""
    import torch

    nvq = _nvq()
    T, D = 6, 64
    g = torch.Generator().manual_seed(4)
    x = ((torch.rand(T, D, generator=g) + 0.5) * (torch.randint(0, 2, (T, D), generator=g) * 2 - 1)).cuda()
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    dy, dh = torch.randn(T, D, generator=g).cuda(), torch.randn(T, D, generator=g).cuda()
    u = torch.randn(T, D, generator=g).sign().cuda() * 2.0 ** -10
    plus, minus = x + u, x - u
    yp, ym = nvq.nvq_rms_norm(plus, w)[0].double(), nvq.nvq_rms_norm(minus, w)[0].double()
    step = plus.double() - minus.double()
    _, h, r = nvq.nvq_rms_norm(x, w, want_rstd=True)
    dx, dw = nvq.nvq_rms_norm_backward(dy, h, w, r, dh=dh)
    want = (dy.double() * (yp - ym)).sum(-1) + (dh.double() * step).sum(-1)
    got = (dx.double() * step).sum(-1)
    # y: 5 roundings each side; third derivative of h / |h|: at most 15 |u|^3 / |h|^3 relative to the row
    rel = float(u.norm(dim=-1).max() / x.norm(dim=-1).min())
    room = (dy.double().abs() * (yp.abs() + ym.abs())).sum(-1) * 6 * ref.U32
    room = room + dy.double().norm(dim=-1) * yp.norm(dim=-1) * 15 * rel ** 3
    (_, _), (e_dx, _) = ref.rms_norm_grad(dy, h, w, r, dh)
    # the derivative is taken at rstd's rounded value
    room = room + (e_dx * step.abs()).sum(-1) + 4 * ref.U32 * (dx.double().abs() * step.abs()).sum(-1)
    assert bool(((got - want).abs() <= room).all()), ((got - want).abs() - room).max()
    # the weight enters linearly
    v = torch.randn(D, generator=g).cuda()
    diff = nvq.nvq_rms_norm(x, w + v)[0].double() - nvq.nvq_rms_norm(x, w - v)[0].double()
    dv = (w + v).double() - (w - v).double()
    room = (dy.double().abs() * (h.double() * r.double()[:, None]).abs() * (w.abs() + v.abs()).double()).sum() * (2 * (T + 12) * ref.U32)
    assert abs(float((dy.double() * diff).sum() - (dw.double() * dv).sum())) <= float(room)


@pytest.mark.parametrize("D", [8, 128, 256, 512, 1024])
def test_rows_that_share_a_wave_do_not_meet(D):
    import torch

    nvq = _nvq()
    T, group = 45, 32 if D >= 32 else 0
    x, _, dy, dh, w = _inputs(T, D, "bfloat16", "float32", seed=11)

    def both(x, dy):
        y, _, r = nvq.nvq_rms_norm(x, w, want_rstd=True)
        codes, scales, _, _ = nvq.nvq_rms_norm_e4m3(x, w, group=group)
        dx, _ = nvq.nvq_rms_norm_backward(dy, x, w, r, dh=dh, want_dw=False)
        return y, r, codes.view(torch.uint8), scales, dx

    clean = both(x, dy)
    x2, dy2 = x.clone(), dy.clone()
    bad = [0, 6, 17, 33, 44]
    x2[bad[0]] = float("nan")
    x2[bad[1], D - 1] = float("inf")
    x2[bad[2]] = 0.0
    dy2[bad[3]] = float("nan")
    dy2[bad[4], 0] = float("inf")
    keep = [t for t in range(T) if t not in bad]
    for a, b in zip(clean, both(x2, dy2)):
        assert torch.equal(a[keep], b[keep])


def test_nothing_to_do_and_the_amax_word():
    import torch

    nvq = _nvq()
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    amax = torch.ones(1, device="cuda")
    y, h, r = nvq.nvq_rms_norm(x, w, residual=x, want_rstd=True, out_amax=amax)
    assert y.shape == (0, 64) and r.shape == (0,) and float(amax) == 0
    codes, scales, _, _ = nvq.nvq_rms_norm_e4m3(x, w, group=32)
    assert codes.shape == (0, 64) and scales.shape == (0, 2)
    dw = torch.ones(64, device="cuda")
    dx, _ = nvq.nvq_rms_norm_backward(x, x, w, r, dw=dw, accumulate=True)
    assert dx.shape == (0, 64) and bool((dw == 1).all())
    nvq.nvq_rms_norm_backward(x, x, w, r, dw=dw)
    assert bool((dw == 0).all())


def test_amax_replaces_the_quantizer_pass():
    import torch

    nvq = _nvq()
    x, res, _, _, w = _inputs(130, 512, "bfloat16", "bfloat16", seed=2)
    amax = torch.zeros(1, device="cuda")
    y, _, _ = nvq.nvq_rms_norm(x, w, residual=res, out_amax=amax)
    a, b = nvq.nvfp4_quantize(y), nvq.nvfp4_quantize(y, amax_in=amax)
    for u, v in zip(a[:3], b[:3]):
        assert torch.equal(u, v)


def test_graph_replays_and_another_stream():
    import torch

    nvq = _nvq()
    x, res, dy, dh, w = _inputs(700, 1024, "bfloat16", "float32", seed=3)
    amax = torch.zeros(1, device="cuda")

    def step():
        y, h, r = nvq.nvq_rms_norm(x, w, residual=res, want_rstd=True, out_amax=amax)
        codes, scales, _, _ = nvq.nvq_rms_norm_e4m3(x, w, residual=res)
        dx, dw = nvq.nvq_rms_norm_backward(dy, h, w, r, dh=dh)
        return y, h, r, amax, codes.view(torch.uint8), scales, dx, dw

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, b in zip(step(), eager):
            assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for rep in range(3):
        amax.fill_(1e9)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b), rep
        step()
        torch.cuda.synchronize()


@pytest.mark.parametrize("group", [128, 32, 0])
@pytest.mark.parametrize("dtype,bits", [("bfloat16", 0x7FC8), ("bfloat16", 0x7FF8), ("bfloat16", -0x0038),
                                        ("float32", 0x7FC80000), ("float32", 0x7FF80003), ("float32", -0x0037FFFE)])
def test_eight_bit_nan_of_any_payload(group, dtype, bits):
    """A NaN keeps its payload through the products; one that looks like a
    midpoint of the format in its low bits is a NaN all the same."""
    import torch

    nvq = _nvq()
    log(f"[norm e4m3 nan] group={group} {dtype} {bits:#x}")
    T, D = 5, 512
    x, res, _, _, w = _inputs(T, D, dtype, "float32", seed=21)
    word = torch.int16 if dtype == "bfloat16" else torch.int32
    clean, clean_scales, _, _ = nvq.nvq_rms_norm_e4m3(x, w, group=group)
    bad = x.clone()
    bad.view(word)[2, 77] = bits
    assert bool(bad[2, 77].isnan())
    codes, scales, _, _ = nvq.nvq_rms_norm_e4m3(bad, w, group=group)
    assert bool(codes[2].float().isnan().all()) and bool(scales[2].isnan().all())
    rest = [0, 1, 3, 4]
    assert torch.equal(codes[rest].view(torch.uint8), clean[rest].view(torch.uint8))
    assert torch.equal(scales[rest], clean_scales[rest])
    # one weight: its groups, and no other
    w2 = w.to(getattr(torch, dtype))
    clean, clean_scales, _, _ = nvq.nvq_rms_norm_e4m3(x, w2, group=group)
    w2 = w2.clone()
    w2.view(word)[200] = bits
    codes, scales, _, _ = nvq.nvq_rms_norm_e4m3(x, w2, group=group)
    n = group or D
    hit = torch.arange(D // n, device="cuda") == 200 // n
    c = codes.view(torch.uint8).reshape(T, D // n, n)
    assert bool(codes.float().reshape(T, D // n, n)[:, hit].isnan().all()) and bool(scales[:, hit].isnan().all())
    assert torch.equal(c[:, ~hit], clean.view(torch.uint8).reshape(T, D // n, n)[:, ~hit])
    assert torch.equal(scales[:, ~hit], clean_scales[:, ~hit])


@pytest.mark.parametrize("D,group", [(512, 128), (512, 32), (4096, 64), (1000, 0), (24, 0)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_both_outputs_of_one_call(D, group, dtype):
    """y beside its codes, as the argument structure allows, with the norm's
    maximum: the bits of two calls."""
    import torch

    nvq = _nvq()
    T = 41
    x, res, _, _, w = _inputs(T, D, dtype, "float32", seed=31)
    amax, amax2 = torch.zeros(1, device="cuda"), torch.full((1,), 5.0, device="cuda")
    y, h, r = nvq.nvq_rms_norm(x, w, residual=res, want_rstd=True, out_amax=amax)
    codes, scales, _, _ = nvq.nvq_rms_norm_e4m3(x, w, residual=res, group=group)
    y2, h2 = torch.zeros_like(y), torch.zeros_like(h)
    codes2, scales2 = torch.zeros_like(codes), torch.zeros_like(scales)
    _, _, r2 = nvq._norm(x, w, 1e-6, res, True, y2, h2, codes2, scales2, group, amax2)
    for a, b in ((y, y2), (h, h2), (r, r2), (codes.view(torch.uint8), codes2.view(torch.uint8)), (scales, scales2), (amax, amax2)):
        assert torch.equal(a, b)
