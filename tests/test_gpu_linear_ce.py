"""The linear cross entropy and its gradient against 64-bit forms: sizes around
the tiles, padded and bad targets, strides, weights of the tokens, both types
of dw, several vocabulary pieces, differences, graphs and streams."""
import pytest

import trainer_reference as ref
from helpers import log

pytestmark = pytest.mark.gpu


def _nvq():
    from qat_nvfp4_quantize_amd import nvq

    return nvq


def _inputs(T, D, V, seed=0, ignore=0, weighted=False, std=0.3):
    import torch

    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + D * 7 + V)
    x = torch.randn(T, D, generator=g).to(torch.bfloat16)
    w = (torch.randn(V, D, generator=g) * std).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g).to(torch.int32)
    if ignore:
        y[::ignore] = -1
    d = torch.randn(T, generator=g) if weighted else torch.full((T,), 1.0 / max(T, 1))
    return x.cuda(), w.cuda(), y.cuda(), d.cuda()


SIZES = [(1, 8, 1), (1, 64, 7), (2, 72, 256), (5, 8, 3000), (16, 256, 1000), (63, 136, 257), (64, 512, 300),
         (65, 64, 513), (255, 200, 255), (256, 128, 512), (257, 320, 1031), (600, 1000, 777), (130, 2056, 130),
         (1000, 64, 2500), (17, 264, 65), (33, 1032, 700), (3, 64, 40000), (40, 520, 33001), (8, 4096, 64),
         (60, 136, 42000), (3000, 72, 4100), (1100, 64, 60001), (300, 1032, 20000),
         (1000, 136, 900), (130, 520, 5000), (16384, 64, 40), (250, 4096, 1000)]


@pytest.mark.parametrize("T,D,V", SIZES)
@pytest.mark.parametrize("scale,ignore,weighted", [(1.0, 0, False), (0.7, 3, True)])
def test_loss_and_gradient_match_64_bits(T, D, V, scale, ignore, weighted):
    import torch

    nvq = _nvq()
    log(f"[ce] T={T} D={D} V={V} scale={scale} ignore={ignore}")
    x, w, y, d = _inputs(T, D, V, ignore=ignore, weighted=weighted)
    (loss, lse, dx, dw), (e_loss, e_lse, e_dx, e_dw) = ref.cross_entropy(x, w, y, scale, d)
    got_loss, got_lse = nvq.nvq_linear_cross_entropy(x, w, y, scale=scale)
    seen = y >= 0
    ref.within(got_loss, loss, e_loss, "loss")
    ref.within(got_lse[seen], lse[seen], e_lse[seen], "lse")
    assert bool((got_loss[~seen] == 0).all())
    got_dx, got_dw = nvq.nvq_linear_cross_entropy_backward(x, w, y, got_lse, d, scale=scale)
    ref.within(got_dx, dx, e_dx, "dx")
    ref.within(got_dw, dw, e_dw + ref.BF16 * (dw.abs() + e_dw), "dw")
    assert bool((got_dx[~seen] == 0).all())
    dw32 = torch.full((V, D), float("nan"), device="cuda")
    only, got32 = nvq.nvq_linear_cross_entropy_backward(x, w, y, got_lse, d, scale=scale, want_dx=False, dw=dw32)
    assert only is None and got32 is dw32
    ref.within(dw32, dw, e_dw + ref.U32 * dw.abs(), "dw fp32")
    # accumulation, one rounding
    nvq.nvq_linear_cross_entropy_backward(x, w, y, got_lse, d, scale=scale, want_dx=False, dw=dw32, accumulate=True)
    ref.within(dw32, 2 * dw, 2 * e_dw + 4 * ref.U32 * dw.abs(), "dw fp32 twice")
    old = got_dw.clone()
    nvq.nvq_linear_cross_entropy_backward(x, w, y, got_lse, d, scale=scale, want_dx=False, dw=got_dw, accumulate=True)
    ref.within(got_dw, old.double() + dw, e_dw + ref.BF16 * ((old.double() + dw).abs() + e_dw), "dw bf16 twice")
    same, none = nvq.nvq_linear_cross_entropy_backward(x, w, y, got_lse, d, scale=scale, want_dw=False)
    assert none is None and torch.equal(same, got_dx)


def test_padded_tokens_may_hold_anything():
    import torch

    nvq = _nvq()
    T, D, V = 300, 96, 700
    x, w, y, d = _inputs(T, D, V, weighted=True)
    y[5:40] = -1
    y[299] = -100
    d[100:110] = 0.0
    loss, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    dx, dw = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d)
    dead = (y < 0) | (d == 0)
    x2, lse2, d2 = x.clone(), lse.clone(), d.clone()
    x2[dead] = float("nan")
    lse2[dead] = float("inf")
    d2[y < 0] = float("nan")
    dx2, dw2 = nvq.nvq_linear_cross_entropy_backward(x2, w, y, lse2, d2)
    assert torch.equal(dw, dw2) and torch.equal(dx, dx2) and bool((dx[dead] == 0).all())
    loss2, lse3 = nvq.nvq_linear_cross_entropy(x2, w, y)
    keep = ~dead
    assert torch.equal(loss2[keep], loss[keep]) and torch.equal(lse3[keep], lse[keep])
    assert bool((loss2[y < 0] == 0).all())
    # nothing counts at all
    none = torch.full_like(y, -1)
    dx, dw = nvq.nvq_linear_cross_entropy_backward(x2, w, none, lse2, d2)
    assert bool((dx == 0).all()) and bool((dw == 0).all())


def test_bad_targets_show_in_the_status():
    import torch

    nvq = _nvq()
    L = nvq.load()
    T, D, V = 70, 64, 300
    x, w, y, d = _inputs(T, D, V)
    ok_loss, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    bad = y.clone()
    bad[3], bad[60] = V, 2 ** 31 - 1
    ws = nvq.workspace(max(L.nvq_linear_cross_entropy_workspace_bytes(T, D, V),
                           L.nvq_linear_cross_entropy_backward_workspace_bytes(T, D, V)), x.device)
    loss, _ = nvq.nvq_linear_cross_entropy(x, w, bad, ws=ws)
    assert nvq.device_status(ws) == nvq.NVQ_STATUS_BAD_TARGET
    assert float(loss[3]) == 0 and float(loss[60]) == 0
    dx, dw = nvq.nvq_linear_cross_entropy_backward(x, w, bad, lse, d, ws=ws)
    assert nvq.device_status(ws) == nvq.NVQ_STATUS_BAD_TARGET
    as_padding = torch.where(bad >= V, -1, bad).to(torch.int32)
    dx2, dw2 = nvq.nvq_linear_cross_entropy_backward(x, w, as_padding, lse, d, ws=ws)
    assert nvq.device_status(ws) == 0
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    nvq.nvq_linear_cross_entropy(x, w, y, ws=ws)
    assert nvq.device_status(ws) == 0


@pytest.mark.parametrize("T", [7, 100])
def test_strided_rows_and_what_lies_between_them(T):
    import torch

    nvq = _nvq()
    D, V = 72, 290
    x, w, y, d = _inputs(T, D, V)
    loss, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    dx, dw = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d)

    def wide(t, pad):
        b = torch.full((t.shape[0], t.shape[1] + 2 * pad), float("nan"), dtype=t.dtype, device="cuda")
        b[:, pad:-pad] = t
        return b, b[:, pad:-pad]

    (_, xs), (_, wsd) = wide(x, 8), wide(w, 24)
    loss2, lse2 = nvq.nvq_linear_cross_entropy(xs, wsd, y)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    (bx, dxs), (bw, dws) = wide(dx, 16), wide(dw, 8)
    nvq.nvq_linear_cross_entropy_backward(xs, wsd, y, lse, d, dx=dxs, dw=dws)
    assert torch.equal(dxs, dx) and torch.equal(dws, dw)
    for b, pad in ((bx, 16), (bw, 8)):
        assert bool(b[:, :pad].isnan().all()) and bool(b[:, -pad:].isnan().all())


def test_extreme_logits():
    import torch

    nvq = _nvq()
    T, D, V = 40, 64, 500
    x, w, y, d = _inputs(T, D, V)
    # logits of thousands: a reference below the maximum would overflow
    (loss, lse, dx, dw), (e_loss, e_lse, e_dx, e_dw) = ref.cross_entropy(x, w, y, 300.0, d)
    got, got_lse = nvq.nvq_linear_cross_entropy(x, w, y, scale=300.0)
    ref.within(got, loss, e_loss, "loss")
    ref.within(got_lse, lse, e_lse, "lse")
    # a negative and a zero scale
    for s in (-0.5, 0.0):
        (loss, lse, dx, dw), (e_loss, e_lse, e_dx, e_dw) = ref.cross_entropy(x, w, y, s, d)
        got, got_lse = nvq.nvq_linear_cross_entropy(x, w, y, scale=s)
        ref.within(got, loss, e_loss, "loss")
        got_dx, got_dw = nvq.nvq_linear_cross_entropy_backward(x, w, y, got_lse, d, scale=s)
        ref.within(got_dx, dx, e_dx, "dx")
        ref.within(got_dw, dw, e_dw + ref.BF16 * (dw.abs() + e_dw), "dw")
    # -inf logits weigh nothing: rows of w that only token 0 and 1 multiply to -inf
    w2, x2 = w.clone(), x.clone()
    w2[100:120, 5] = float("-inf")
    x2[:, 5] = 1.0
    y2 = torch.where((y >= 100) & (y < 120), 7, y).to(torch.int32)
    keep = torch.ones(V, dtype=torch.bool, device="cuda")
    keep[100:120] = False
    moved = torch.where(y2 >= 120, y2 - 20, y2).to(torch.int32)
    (loss, lse, _, _), (e_loss, e_lse, _, _) = ref.cross_entropy(x2, w2[keep], moved, 1.0)
    got, got_lse = nvq.nvq_linear_cross_entropy(x2, w2, y2)
    ref.within(got, loss, e_loss, "loss beside -inf")
    ref.within(got_lse, lse, e_lse, "lse beside -inf")
    # a NaN token stays alone
    x3 = x.clone()
    x3[11, 0] = float("nan")
    clean, _ = nvq.nvq_linear_cross_entropy(x, w, y)
    got, got_lse = nvq.nvq_linear_cross_entropy(x3, w, y)
    rest = torch.arange(T, device="cuda") != 11
    assert bool(got[11].isnan()) and bool(got_lse[11].isnan()) and torch.equal(got[rest], clean[rest])


def test_weights_of_very_different_size_and_non_finite_ones():
    import torch

    nvq = _nvq()
    T, D, V = 90, 64, 300
    x, w, y, _ = _inputs(T, D, V)
    d = torch.logspace(-30, 20, T, device="cuda") * torch.where(torch.arange(T, device="cuda") % 2 == 0, 1.0, -1.0)
    (_, _, dx, dw), (_, _, e_dx, e_dw) = ref.cross_entropy(x, w, y, 1.0, d)
    _, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    got_dx, got_dw = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d)
    # entries under 2^-126 of the largest weight leave fp32's normal numbers
    under = float(d.abs().max()) * 2.0 ** -126 * 300
    ref.within(got_dx, dx, e_dx + under, "dx")
    ref.within(got_dw, dw, e_dw + ref.BF16 * (dw.abs() + e_dw) + under, "dw")
    # default weights are ones
    one = torch.ones(T, device="cuda")
    a, b = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse), nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, one)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one[4] = float("inf")
    got_dx, _ = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, one)
    rest = torch.arange(T, device="cuda") != 4
    assert torch.equal(got_dx[rest], a[0][rest]) and not bool(got_dx[4].isfinite().any())


@pytest.mark.parametrize("T,D,V,same", [(700, 96, 2000, False), (300, 64, 300, False), (2600, 64, 40, True), (4500, 512, 20000, True),
                                        (1000, 264, 40000, False)])
def test_target_terms_keep_their_weights(T, D, V, same):
    """With w = 0 every probability is 1 / V and dw is known exactly.  Where
    weights differ, a target's own term is good to 2^-15 and the fp32 sum's
    rounding (three addends a token), not to bf16's rounding of the weighted
    state; same: the targets are one word, whose terms would all be off the same
    way (by 2.2e-3: 0.7 times 1 + 2^-7)."""
    import torch

    nvq = _nvq()
    x, w, y, d = _inputs(T, D, V, weighted=True, ignore=0 if same else 5)
    w = torch.zeros_like(w)
    if same:
        y = torch.full_like(y, V - 3)
        x = (torch.sign(x.float()) * (1 + 2.0 ** -7)).to(torch.bfloat16)
        x[:] = x[0]
        d = torch.full_like(d, 0.7)
        d[T // 2] = 1.0
    _, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    _, got = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d, want_dx=False, dw=torch.empty(V, D, device="cuda"))
    live = y >= 0
    term = (d.double()[:, None] * x.double())[live]
    own = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, y[live].long(), term)
    own_mag = torch.zeros_like(own).index_add_(0, y[live].long(), term.abs())
    dw = term.sum(0) / V - own
    total = term.abs().sum(0) / V
    fp32 = (T + 16) * ref.U32
    room = own_mag * (2.0 ** -15 + 3 * fp32 + 1.0 / V * (2 * ref.BF16)) + total * (2 * ref.BF16 + 2.0 ** -15 + fp32 + 1e-5)
    ref.within(got, dw, room + 2 * ref.U32 * dw.abs(), "dw")


def test_several_pieces_of_the_vocabulary():
    import torch

    nvq = _nvq()
    T, D, V = 16300, 64, 40001
    x, w, y, d = _inputs(T, D, V, ignore=7, weighted=True)
    L = nvq.load()
    # c of the whole vocabulary would not fit what the workspace holds of it
    assert L.nvq_linear_cross_entropy_backward_workspace_bytes(T, D, V) < 2 * T * V
    got_loss, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    got_dx, got_dw = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d)
    rows = torch.arange(0, T, 9, device="cuda")
    (loss, _, dx, _), (e_loss, _, e_dx, _) = ref.cross_entropy(x[rows], w, y[rows], 1.0, d[rows])
    ref.within(got_loss[rows], loss, e_loss, "loss")
    # c is rounded after division by the largest weight of the whole call, which changes no bound
    ref.within(got_dx[rows], dx, e_dx, "dx")
    # dw of the words at the pieces' ends and some between, from the exact probabilities
    words = torch.cat([torch.arange(k, min(k + 40, V), device="cuda") for k in (0, 16360, 16384, 32760, 39990)])
    live = y >= 0
    z = x.double() @ w[words].double().T
    c = torch.exp(z - lse.double()[:, None]) - (y[:, None] == words[None]).double()
    c = torch.where(live[:, None], c * d.double()[:, None], 0.0)
    dw = c.T @ x.double()
    mag = c.abs().T @ x.double().abs()
    ref.within(got_dw[words], dw, mag * (2 * ref.BF16 + 1e-4) + ref.BF16 * dw.abs(), "dw")


def test_gradient_against_differences_of_the_loss():
    """sum(dloss loss) at x + u and x - u, both exact in bf16: the difference is
    2 <dx, u> up to the third derivative, at most (2 max|u w|)^3 / 3 a token."""
    import torch

    nvq = _nvq()
    T, D, V = 50, 32, 400
    x, w, y, d = _inputs(T, D, V, weighted=True)
    x = (x * 4).round().clamp(-12, 12) / 4  # multiples of 1/4 up to 3: x +- 1/64 stays within 8 bits
    g = torch.Generator().manual_seed(3)
    u = ((torch.randint(0, 2, (T, D), generator=g) * 2 - 1) / 64.0).to(torch.bfloat16).cuda()
    plus, minus = (x.float() + u.float()).to(torch.bfloat16), (x.float() - u.float()).to(torch.bfloat16)
    x = x.to(torch.bfloat16)
    step = (plus.double() - minus.double()) / 2
    step = torch.where((plus.double() + minus.double()) / 2 == x.double(), step, 0.0)
    plus, minus = (x.double() + step).to(torch.bfloat16), (x.double() - step).to(torch.bfloat16)
    assert torch.equal(plus.double() - x.double(), step) and float(step.abs().max()) > 0
    a, b = nvq.nvq_linear_cross_entropy(plus, w, y)[0].double(), nvq.nvq_linear_cross_entropy(minus, w, y)[0].double()
    _, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    dx, _ = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d, want_dw=False)
    _, (e_a, _, _, _) = ref.cross_entropy(plus, w, y, 1.0)
    _, (_, _, e_dx, _) = ref.cross_entropy(x, w, y, 1.0, d)
    third = (2 * (step @ w.double().T).abs().amax(-1)) ** 3 / 3
    room = d.double().abs() * (2 * e_a + third) + 2 * (e_dx * step.abs()).sum(-1)
    off = (d.double() * (a - b) - 2 * (dx.double() * step).sum(-1)).abs()
    assert bool((off <= room).all()), float((off - room).max())
    # a sum over the tokens for w: the words' rows move by multiples of 1/256
    v = torch.zeros_like(w)
    w = (w * 16).round() / 16
    v[:, 3] = 1.0 / 64
    p, m = (w.float() + v.float()).to(torch.bfloat16), (w.float() - v.float()).to(torch.bfloat16)
    ok = ((p.double() + m.double()) / 2 == w.double())[:, 3]
    v[~ok] = 0
    p, m = (w.double() + v.double()).to(torch.bfloat16), (w.double() - v.double()).to(torch.bfloat16)
    w = w.to(torch.bfloat16)
    a, b = nvq.nvq_linear_cross_entropy(x, p, y)[0].double(), nvq.nvq_linear_cross_entropy(x, m, y)[0].double()
    _, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    dw32 = torch.empty(V, D, device="cuda")
    nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d, want_dx=False, dw=dw32)
    _, (e_a, _, _, e_dw) = ref.cross_entropy(x, w, y, 1.0, d)
    third = (2 * (x.double() @ v.double().T).abs().amax(-1)) ** 3 / 3
    room = (d.double().abs() * (2 * 1.1 * e_a + third)).sum() + 2 * ((e_dw + ref.U32 * dw32.abs()) * v.double().abs()).sum()
    off = ((d.double() * (a - b)).sum() - 2 * (dw32.double() * v.double()).sum()).abs()
    assert float(off) <= float(room), (float(off), float(room))


def test_no_tokens():
    import torch

    nvq = _nvq()
    x, w, y, d = _inputs(0, 64, 100)
    loss, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    assert loss.shape == (0,) and lse.shape == (0,)
    dw = torch.ones(100, 64, device="cuda")
    dx, _ = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d, dw=dw, accumulate=True)
    assert dx.shape == (0, 64) and bool((dw == 1).all())
    nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d, dw=dw)
    assert bool((dw == 0).all())


def test_graphs_streams_and_a_shared_workspace():
    import torch

    nvq = _nvq()
    L = nvq.load()
    sets = [_inputs(130, 128, 700, seed=1, weighted=True), _inputs(333, 128, 700, seed=2, ignore=4)]
    ws = nvq.workspace(max(max(L.nvq_linear_cross_entropy_workspace_bytes(x.shape[0], 128, 700),
                               L.nvq_linear_cross_entropy_backward_workspace_bytes(x.shape[0], 128, 700))
                           for x, _, _, _ in sets), "cuda")

    def step(s, ws):
        x, w, y, d = s
        loss, lse = nvq.nvq_linear_cross_entropy(x, w, y, ws=ws)
        return loss, lse, *nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d, ws=ws)

    eager = [[t.clone() for t in step(s, None)] for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s, e in zip(sets, eager):
            for a, b in zip(step(s, ws), e):
                assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(s, ws)
        graphs.append((g, outs))
    for rep in range(3):
        for (g, outs), e in zip(graphs, eager):
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, e):
                assert torch.equal(a, b), rep
        step(sets[rep % 2], ws)  # eager work over the same workspace between the replays
        torch.cuda.synchronize()


@pytest.mark.parametrize("T,V", [(40, 500), (300, 700), (300, 30000), (48, 70000)])
@pytest.mark.parametrize("weights", ["equal", "powers of two", "any"])
def test_each_product_of_dw_is_rounded_once(T, V, weights):
    """Every token has columns of its own, so an element of dw is one product c
    dloss x: off by one rounding to bf16, of c and the weight together, whatever
    the weights are (a second one, of the weighted state, would make it up to
    2^-7), and by c's own error.  A target's own is good to 2^-15."""
    import torch

    nvq = _nvq()
    log(f"[ce once] T={T} V={V} {weights}")
    D = 8 * T
    x, w, y, _ = _inputs(T, D, V, seed=6)
    own = torch.arange(D, device="cuda") // 8 == torch.arange(T, device="cuda")[:, None]
    x = torch.where(own, x, 0.0)
    g = torch.Generator().manual_seed(T)
    d = {"equal": torch.full((T,), 0.3), "any": torch.rand(T, generator=g) * 0.9 + 0.1,
         "powers of two": 0.3 * 2.0 ** torch.randint(-9, 1, (T,), generator=g)}[weights]
    d = (d * (torch.randint(0, 2, (T,), generator=g) * 2 - 1)).cuda()
    _, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    _, got = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d, want_dx=False, dw=torch.empty(V, D, device="cuda"))
    part = w.reshape(V, T, 8)  # [word, token, its columns]
    xs = x.reshape(T, T, 8).diagonal(dim1=0, dim2=1).T  # [token, its columns]
    off, worst = 0.0, 0.0
    for v0 in range(0, V, 10000):
        words = torch.arange(v0, min(v0 + 10000, V), device="cuda")
        p = part[words].double()
        z = (p * xs.double()).sum(-1)  # [word, token]
        dz = 9 * ref.ADD * (p * xs.double()).abs().sum(-1)
        prob = torch.exp(z - lse.double())
        hit = words[:, None] == y
        c = prob - hit.double()
        rel = dz + 8 * ref.U32 * (z.abs() + lse.double().abs()) + 4 * ref.U32  # of the given lse
        want = (c * d.double())[:, :, None] * xs.double()
        e_c = prob * rel + 4 * ref.U32 * c.abs()
        e_c = e_c + (c.abs() + e_c) * torch.where(hit & (weights == "any"), 2.0 ** -15, ref.BF16)
        room = (e_c * d.double().abs())[:, :, None] * xs.double().abs()
        room = (room + 12 * ref.U32 * want.abs()).reshape(len(words), D)
        ref.within(got[words], want.reshape(len(words), D), room, "dw")


def test_weighted_dx_keeps_its_targets_term():
    """w has one element in each target's row and none elsewhere: an element of
    dx is one product c dloss w.  The target's own is as good as dx's rounding
    lets it be, the others' are off by one more of c and the weight."""
    import torch

    nvq = _nvq()
    T, V = 96, 3000
    D = T
    x, w, y, _ = _inputs(T, D, V, seed=8, weighted=True)
    g = torch.Generator().manual_seed(5)
    y = torch.randperm(V, generator=g)[:T].to(torch.int32).cuda()
    w = torch.zeros_like(w)
    w[y.long(), torch.arange(T, device="cuda")] = (torch.rand(T, generator=g) + 0.5).to(torch.bfloat16).cuda()
    d = (torch.rand(T, generator=g) + 0.01).cuda()
    _, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    dx, _ = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d, want_dw=False)
    wd = w[y.long(), torch.arange(T, device="cuda")].double()
    z = x.double() * wd  # [token, target of column]
    hit = torch.eye(T, dtype=torch.bool, device="cuda")
    prob = torch.exp(z - lse.double()[:, None])
    c = prob - hit.double()
    rel = 4 * ref.ADD * z.abs() + 8 * ref.U32 * (z.abs() + lse.double()[:, None].abs()) + 4 * ref.U32
    want = c * d.double()[:, None] * wd
    e_c = prob * rel + 4 * ref.U32 * c.abs()
    e_c = e_c + (c.abs() + e_c) * torch.where(hit, 2.0 ** -15, ref.BF16)
    room = e_c * d.double()[:, None] * wd + 12 * ref.U32 * want.abs()
    ref.within(dx, want, room + ref.BF16 * (want.abs() + room), "dx")


@pytest.mark.parametrize("T,V", [(20, 300), (300, 5000)])
def test_losses_of_sure_tokens(T, V):
    """Logits of thousands whose target leads by up to forty: the loss is the
    others' share, not the difference of two large numbers.  It is never
    negative, and off by the sums of exponentials' roundings (130, as the bound
    of the log-sum-exp counts them), three of its own, and the logits' own error
    times that share."""
    import torch

    nvq = _nvq()
    log(f"[ce sure] T={T} V={V}")
    D = 8 + -(-T // 8) * 8
    g = torch.Generator().manual_seed(9)
    t = torch.arange(T)
    w = torch.randint(-2, 3, (V, D), generator=g).to(torch.bfloat16)
    y = torch.randperm(V, generator=g)[:T].to(torch.int32)
    x = torch.zeros(T, D)
    x[:, 0] = 32.0 + t % 4          # times 64: what all logits of half the vocabulary have in common
    x[t, 8 + t] = (t % 11) / 32.0   # times 120: the target's lead
    x = x.to(torch.bfloat16)
    w[:V // 2, 0] = 64.0
    w[y.long(), 0] = 64.0
    w[y.long(), 8 + t] = 120.0
    x, w, y = x.cuda(), w.cuda(), y.cuda()
    loss, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    # every logit is exact in fp32: two products of few bits
    z = x.double() @ w.double().T
    assert torch.equal(z, z.float().double()) and float(z.max()) > 2000
    at = z.gather(1, y.long()[:, None])
    want = torch.log1p(torch.exp(z - at).sum(-1) - 1.0)
    share = 1 - torch.exp(-want.clamp(min=0))
    # of a logit: its product with log2(e), and the subtraction
    arg = 4 * ref.U32 * z.abs().amax(-1)
    room = 130 * ref.U32 + 4 * ref.U32 * want.abs() + share * arg
    assert bool((loss >= 0).all())
    ref.within(loss, want, room, "loss")


# what the kernel for few tokens does not take: as quarters of tiles, as whole
# ones, as whole ones in one column
TILED = [(300, 5000), (520, 15001), (250, 40001)]
TILED_SIZES = [(255, 64, 16385), (257, 72, 5120), (256, 128, 25599), (513, 64, 11009), (130, 2056, 8193), (600, 1000, 8000),
               (64, 264, 41000), (65, 64, 33000)]


@pytest.mark.parametrize("T,D,V", TILED_SIZES)
@pytest.mark.parametrize("scale,ignore,weighted", [(1.0, 0, False), (0.7, 3, True)])
def test_tiled_loss_and_gradient_match_64_bits(T, D, V, scale, ignore, weighted):
    test_loss_and_gradient_match_64_bits(T, D, V, scale, ignore, weighted)


@pytest.mark.parametrize("T,V", TILED)
def test_tiled_strided_rows(T, V):
    import torch

    nvq = _nvq()
    log(f"[ce tiled strided] T={T} V={V}")
    D = 72
    x, w, y, d = _inputs(T, D, V, ignore=7, weighted=True)
    loss, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    dx, dw = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d)

    def wide(t, pad):
        b = torch.full((t.shape[0], t.shape[1] + 2 * pad), float("nan"), dtype=t.dtype, device="cuda")
        b[:, pad:-pad] = t
        return b, b[:, pad:-pad]

    (_, xs), (_, wsd) = wide(x, 8), wide(w, 24)
    loss2, lse2 = nvq.nvq_linear_cross_entropy(xs, wsd, y)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    for dtype in (torch.bfloat16, torch.float32):
        (bx, dxs), (bw, dws) = wide(dx, 16), wide(dw.to(dtype), 8)
        for accumulate in (False, True):
            dws[:] = 0.0 if accumulate else 7.0
            nvq.nvq_linear_cross_entropy_backward(xs, wsd, y, lse, d, dx=dxs, dw=dws, accumulate=accumulate)
            assert torch.equal(dxs, dx) and torch.equal(dws.to(torch.bfloat16), dw)
            for b, pad in ((bx, 16), (bw, 8)):
                assert bool(b[:, :pad].isnan().all()) and bool(b[:, -pad:].isnan().all())


@pytest.mark.parametrize("T,V", TILED)
def test_tiled_padded_tokens_and_bad_targets(T, V):
    import torch

    nvq = _nvq()
    L = nvq.load()
    log(f"[ce tiled padded] T={T} V={V}")
    D = 96
    x, w, y, d = _inputs(T, D, V, weighted=True)
    y[5:40] = -1
    y[T - 1] = -100
    loss, lse = nvq.nvq_linear_cross_entropy(x, w, y)
    dx, dw = nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d)
    assert bool((loss[y < 0] == 0).all()) and bool((dx[y < 0] == 0).all())
    bad = y.clone()
    bad[7], bad[T - 1], bad[39] = V, 2 ** 31 - 1, V + 255
    x2, lse2 = x.clone(), lse.clone()
    x2[y < 0] = float("nan")
    lse2[y < 0] = float("nan")
    ws = nvq.workspace(max(L.nvq_linear_cross_entropy_workspace_bytes(T, D, V),
                           L.nvq_linear_cross_entropy_backward_workspace_bytes(T, D, V)), x.device)
    live = y >= 0
    for targets, status in ((bad, nvq.NVQ_STATUS_BAD_TARGET), (y, 0)):
        ws.fill_(255)
        loss2, lse3 = nvq.nvq_linear_cross_entropy(x2, w, targets, ws=ws)
        assert nvq.device_status(ws) == status
        assert torch.equal(loss2, loss) and torch.equal(lse3[live], lse[live]) and bool(lse3[~live].isnan().all())
        ws.fill_(255)
        dx2, dw2 = nvq.nvq_linear_cross_entropy_backward(x2, w, targets, lse2, d, ws=ws)
        assert nvq.device_status(ws) == status
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("T,V", TILED)
def test_tiled_extreme_logits(T, V):
    import torch

    nvq = _nvq()
    log(f"[ce tiled extreme] T={T} V={V}")
    D = 64
    x, w, y, d = _inputs(T, D, V)
    for scale in (300.0, -0.5, 0.0):
        (loss, lse, dx, dw), (e_loss, e_lse, e_dx, e_dw) = ref.cross_entropy(x, w, y, scale, d)
        got, got_lse = nvq.nvq_linear_cross_entropy(x, w, y, scale=scale)
        ref.within(got, loss, e_loss, "loss")
        ref.within(got_lse, lse, e_lse, "lse")
        if scale != 300.0:
            got_dx, got_dw = nvq.nvq_linear_cross_entropy_backward(x, w, y, got_lse, d, scale=scale)
            ref.within(got_dx, dx, e_dx, "dx")
            ref.within(got_dw, dw, e_dw + ref.BF16 * (dw.abs() + e_dw), "dw")
    # words of logit -inf weigh nothing: some, a whole block of 128 words, the last ones
    keep = torch.ones(V, dtype=torch.bool, device="cuda")
    keep[100:120] = False
    keep[256:512] = False
    keep[V - 3:] = False
    w2, x2 = w.clone(), x.clone()
    w2[~keep, 5] = float("-inf")
    x2[:, 5] = 1.0
    y2 = torch.where(keep[y.long()], y, 7).to(torch.int32)
    moved = (torch.cumsum(keep, 0) - 1)[y2.long()].to(torch.int32)
    (loss, lse, _, _), (e_loss, e_lse, _, _) = ref.cross_entropy(x2, w2[keep], moved, 1.0)
    got, got_lse = nvq.nvq_linear_cross_entropy(x2, w2, y2)
    ref.within(got, loss, e_loss, "loss beside -inf")
    ref.within(got_lse, lse, e_lse, "lse beside -inf")
    # nothing but -inf: the log-sum-exp of an empty sum, and no loss
    x3 = x.clone()
    x3[0], x3[T - 1] = 0.0, 0.0
    x3[0, 0], x3[T - 1, 0] = float("-inf"), float("-inf")
    w3 = w.clone()
    w3[:, 0] = w3[:, 0].abs() + 0.5
    base, base_lse = nvq.nvq_linear_cross_entropy(x, w3, y)
    got, got_lse = nvq.nvq_linear_cross_entropy(x3, w3, y)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[0] = rest[T - 1] = False
    assert bool((got_lse[~rest] == float("-inf")).all()) and bool(got[~rest].isnan().all())
    assert torch.equal(got[rest], base[rest]) and torch.equal(got_lse[rest], base_lse[rest])
    # NaN and +inf stay with their tokens
    x4 = x.clone()
    x4[11, 0] = float("nan")
    x4[T - 2] = 0.0
    x4[T - 2, 0] = float("inf")
    got, got_lse = nvq.nvq_linear_cross_entropy(x4, w3, y)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[11] = rest[T - 2] = False
    assert bool(got[~rest].isnan().all()) and bool(got_lse[~rest].isnan().all())
    assert torch.equal(got[rest], base[rest]) and torch.equal(got_lse[rest], base_lse[rest])


def test_tiled_graphs_streams_and_a_shared_workspace():
    import torch

    nvq = _nvq()
    L = nvq.load()
    D = 128
    sets = [_inputs(T, D, V, seed=k, weighted=k == 1, ignore=4 * (k % 2)) for k, (T, V) in enumerate(TILED)]
    ws = nvq.workspace(max(max(L.nvq_linear_cross_entropy_workspace_bytes(T, D, V),
                               L.nvq_linear_cross_entropy_backward_workspace_bytes(T, D, V)) for T, V in TILED), "cuda")

    def step(s, ws):
        x, w, y, d = s
        loss, lse = nvq.nvq_linear_cross_entropy(x, w, y, ws=ws)
        return loss, lse, *nvq.nvq_linear_cross_entropy_backward(x, w, y, lse, d, ws=ws)

    eager = [[t.clone() for t in step(s, None)] for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s, e in zip(sets, eager):
            for a, b in zip(step(s, ws), e):
                assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(s, ws)
        graphs.append((g, outs))
    for rep in range(3):
        for (g, outs), e in zip(graphs, eager):
            for t in outs:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, e):
                assert torch.equal(a, b), rep
        step(sets[rep % 3], ws)  # eager work over the same workspace between the replays
        torch.cuda.synchronize()
