"""The global gradient norm and clipping against 64-bit forms."""
import math

import pytest

import trainer_reference as ref
from helpers import log

pytestmark = pytest.mark.gpu


def _nvq():
    from qat_nvfp4_quantize_amd import nvq

    return nvq


def _tensors(sizes, seed=0, big=1.0):
    import torch

    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n, generator=g) * big
        out.append(t.to(torch.bfloat16 if i % 2 else torch.float32).cuda())
    return out


def _norm64(tensors):
    return math.sqrt(sum(float(t.double().square().sum()) for t in tensors))


def _check_norm(got, want):
    # rounded once from fp64 sums
    assert abs(float(got) - want) <= (ref.U32 + 1e-12) * want, (float(got), want)


LISTS = [[1], [1, 1], [7], [8], [9, 0, 15], [4096], [16385, 3], [100000, 17, 0, 1, 65536], [33] * 300, [2048 * 8 + 5] * 7,
         [5000000, 12], [4 * 2048, 8 * 2048, 8 * 2048 + 1]]


@pytest.mark.parametrize("sizes", LISTS, ids=[str(i) for i in range(len(LISTS))])
@pytest.mark.parametrize("ratio", [0.3, 2.0])
def test_norm_and_clipping(sizes, ratio):
    import torch

    nvq = _nvq()
    log(f"[clip] {len(sizes)} tensors, {sum(sizes)} elements, ratio {ratio}")
    grads = _tensors(sizes)
    want = _norm64(grads)
    _check_norm(nvq.nvq_grad_norm(grads), want)
    most = ratio * want
    outs = [torch.full_like(t, float("nan")) for t in grads]
    _check_norm(nvq.nvq_clip_grad_norm(grads, most, out=outs), want)
    coef = min(1.0, float(torch.tensor(most)) / want)
    for t, o in zip(grads, outs):
        if ratio > 1:
            assert torch.equal(t, o)
            continue
        e = ref.round_error(t.dtype)
        v = t.double() * coef
        ref.within(o, v, (3 * ref.U32 + e) * v.abs() + (2.0 ** -133 if t.dtype == torch.bfloat16 else 2.0 ** -149), "clipped")
    mine = [t.clone() for t in grads]
    norm = nvq.nvq_clip_grad_norm(mine, most)
    _check_norm(norm, want)
    for a, b in zip(mine, outs):
        assert torch.equal(a, b)
    if ratio < 1:
        assert abs(float(nvq.nvq_grad_norm(mine)) / float(torch.tensor(most)) - 1) <= 2 * ref.BF16


def test_views_at_any_offset_and_their_neighbours():
    """Slices of one buffer, as gradient buckets hold them, at every alignment;
    outputs at other alignments than the inputs."""
    import torch

    nvq = _nvq()
    for dtype in (torch.bfloat16, torch.float32):
        g = torch.Generator().manual_seed(8)
        flat = torch.randn(40000, generator=g).to(dtype).cuda()
        out = torch.full((40100,), 5.0, dtype=dtype, device="cuda")
        sizes = [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 1001, 16391, 20000]
        grads, outs, at = [], [], 0
        for i, n in enumerate(sizes):
            grads.append(flat[at:at + n])
            outs.append(out[at + 3 + 2 * i:at + 3 + 2 * i + n])
            at += n + (i % 3)
        want = _norm64(grads)
        before = flat.clone()
        _check_norm(nvq.nvq_clip_grad_norm(grads, 0.25 * want, out=outs), want)
        assert torch.equal(flat, before)
        for t, o in zip(grads, outs):
            v = t.double() * 0.25
            ref.within(o, v, (4 * ref.U32 + ref.round_error(dtype)) * v.abs() + 2.0 ** -133, "clipped")
        touched = torch.zeros(40100, dtype=torch.bool, device="cuda")
        at = 0
        for i, n in enumerate(sizes):
            touched[at + 3 + 2 * i:at + 3 + 2 * i + n] = True
            at += n + (i % 3)
        assert bool((out[~touched] == 5).all())
        keep = torch.ones(40000, dtype=torch.bool, device="cuda")
        at = 0
        for i, n in enumerate(sizes):
            keep[at:at + n] = False
            at += n + (i % 3)
        nvq.nvq_clip_grad_norm(grads, 0.25 * want)
        assert torch.equal(flat[keep], before[keep])


def test_size_of_squares_and_non_finite_norms():
    import torch

    nvq = _nvq()
    ws = nvq.workspace(1 << 20, "cuda")
    for size in (1e30, 1e-30):
        grads = _tensors([1000, 333, 5], big=size)
        want = _norm64(grads)
        _check_norm(nvq.nvq_grad_norm(grads, ws=ws), want)
        assert nvq.device_status(ws) == 0
    for bad in (float("nan"), float("inf")):
        grads = _tensors([1000, 333, 5])
        grads[1][7] = bad
        before = [t.clone() for t in grads]
        outs = [torch.zeros_like(t) for t in grads]
        norm = nvq.nvq_clip_grad_norm(grads, 1e-3, out=outs, ws=ws)
        assert nvq.device_status(ws) == nvq.NVQ_STATUS_NONFINITE and not math.isfinite(float(norm))
        nvq.nvq_clip_grad_norm(grads, 1e-3, ws=ws)
        for a, b, c in zip(grads, before, outs):
            assert torch.equal(a.nan_to_num(3.0), b.nan_to_num(3.0)) and torch.equal(c.nan_to_num(3.0), b.nan_to_num(3.0))
    # a zero bound, zero gradients, infinity, nothing
    grads = _tensors([100, 50])
    nvq.nvq_clip_grad_norm(grads, 0.0)
    assert all(bool((t == 0).all()) for t in grads)
    assert float(nvq.nvq_clip_grad_norm(grads, 1.0)) == 0 and all(bool((t == 0).all()) for t in grads)
    grads = _tensors([100, 50])
    before = [t.clone() for t in grads]
    nvq.nvq_clip_grad_norm(grads, float("inf"))
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    assert float(nvq.nvq_grad_norm([])) == 0 and float(nvq.nvq_clip_grad_norm([], 1.0)) == 0


def test_large_tensor_past_32_bits_of_bytes():
    import torch

    nvq = _nvq()
    n = (1 << 31) + 12345  # bf16: 4.3 GB
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[0], t[n // 2], t[-1] = 3.0, 4.0, 12.0
    assert float(nvq.nvq_grad_norm([t])) == 13.0
    assert float(nvq.nvq_clip_grad_norm([t], 6.5)) == 13.0
    assert float(t[0]) == 1.5 and float(t[n // 2]) == 2.0 and float(t[-1]) == 6.0
    assert float(nvq.nvq_grad_norm([t])) == 6.5


def test_refusals():
    import torch

    nvq = _nvq()
    a = torch.zeros(100, device="cuda")
    for bad in ([a.cpu()], [a, a.cpu()], [a.half()], [torch.zeros(4, 4, device="cuda").t()[1:]], [a.double()]):
        with pytest.raises(ValueError):
            nvq.nvq_grad_norm(bad)
    with pytest.raises(ValueError):
        nvq.nvq_clip_grad_norm([a, a], 1.0)
    with pytest.raises(ValueError):
        nvq.nvq_clip_grad_norm([a[:60], a[50:]], 1.0)
    with pytest.raises(ValueError):
        nvq.nvq_clip_grad_norm([a.clone(), a.clone()], 1.0, out=[a, a])
    assert float(nvq.nvq_grad_norm([a + 1, a + 1])) == pytest.approx(math.sqrt(200))
    for max_norm in (-1.0, float("nan")):
        with pytest.raises(nvq.NvqError):
            nvq.nvq_clip_grad_norm([a], max_norm)
    with pytest.raises(nvq.NvqError):
        nvq.nvq_clip_grad_norm([a], 1.0, out=[a[:50]])
    with pytest.raises(nvq.NvqError):
        nvq.nvq_clip_grad_norm([a], 1.0, out=[])
    b = a + 1
    with pytest.raises(nvq.NvqError):
        nvq.nvq_clip_grad_norm([a, b], 1.0, out=[b, a])
    with pytest.raises(nvq.NvqError):
        nvq.nvq_clip_grad_norm([a[:50], b[:50]], 1.0, out=[b[50:], a[40:90]])
    assert bool((a == 0).all()) and bool((b == 1).all())


def test_graph_replays_over_changing_gradients():
    import torch

    nvq = _nvq()
    grads = nvq.TensorList(_tensors([70000, 33, 20000, 8] * 40))
    ws = nvq.workspace(nvq.load().nvq_grad_norm_workspace_bytes(grads._ref), "cuda")
    start = [t.clone() for t in grads.tensors]

    def reset(k):
        for t, s in zip(grads.tensors, start):
            t.copy_(s * k)

    nvq.nvq_clip_grad_norm(grads, 10.0, ws=ws)  # warm
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm = nvq.nvq_clip_grad_norm(grads, 10.0, ws=ws)
    for k in (1.0, 2.0, 0.5, 2.0 ** -12):
        reset(k)
        g.replay()
        torch.cuda.synchronize()
        got, n = [t.clone() for t in grads.tensors], float(norm)
        reset(k)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            m = float(nvq.nvq_clip_grad_norm(grads, 10.0, ws=ws))
        torch.cuda.current_stream().wait_stream(side)
        assert n == m and all(torch.equal(a, b) for a, b in zip(got, grads.tensors)), k


def test_a_norm_past_the_largest_number_scales_nothing():
    """The norm is handed out in fp32: where it is infinite there, although no
    gradient is, nothing is scaled and the status says so."""
    import torch

    nvq = _nvq()
    ws = nvq.workspace(1 << 20, "cuda")
    for dtype in (torch.float32, torch.bfloat16):
        grads = [torch.full((37,), 3e38, device="cuda").to(dtype), torch.ones(500, device="cuda", dtype=dtype)]
        before = [t.clone() for t in grads]
        outs = [torch.zeros_like(t) for t in grads]
        assert math.isinf(float(nvq.nvq_grad_norm(grads, ws=ws))) and nvq.device_status(ws) == nvq.NVQ_STATUS_NONFINITE
        assert math.isinf(float(nvq.nvq_clip_grad_norm(grads, 1.0, out=outs, ws=ws)))
        assert nvq.device_status(ws) == nvq.NVQ_STATUS_NONFINITE
        nvq.nvq_clip_grad_norm(grads, 1.0, ws=ws)
        assert nvq.device_status(ws) == nvq.NVQ_STATUS_NONFINITE
        for a, b, c in zip(grads, before, outs):
            assert torch.equal(a, b) and torch.equal(c, b)
        # the largest norm that is a number still clips
        grads = [torch.full((1,), 3e38, device="cuda").to(dtype)]
        norm = float(nvq.nvq_clip_grad_norm(grads, 1.0, ws=ws))
        assert math.isfinite(norm) and nvq.device_status(ws) == 0
        assert abs(float(grads[0][0]) - 1.0) <= 2 * ref.round_error(dtype)


@pytest.mark.parametrize("offset", [0, 1])
def test_gradients_that_are_not_scaled_come_bit_by_bit(offset):
    """NaN payloads, signalling ones and their signs among them, into aligned and
    unaligned results, in vectors and in the elements beside them."""
    import torch

    nvq = _nvq()
    for dtype, word, specials in (
            (torch.bfloat16, torch.int16, [0x7FC8, 0x7F81, -0x007F, -0x0001, 0x7F80, -0x0080, 0x0001, -0x8000]),
            (torch.float32, torch.int32, [0x7FC80000, 0x7F800001, -0x007FFFFF, -1, 0x7F800000, -0x00800000, 1, -0x80000000])):
        g = torch.Generator().manual_seed(2)
        t = torch.randn(1003, generator=g).to(dtype).cuda()
        bits = t.view(word)
        bits[:8] = torch.tensor(specials, dtype=word)
        bits[500:508] = torch.tensor(specials, dtype=word)
        bits[-8:] = torch.tensor(specials, dtype=word)
        out = torch.zeros(1003 + offset, dtype=dtype, device="cuda")[offset:]
        nvq.nvq_clip_grad_norm([t], 1e-3, out=[out])
        assert torch.equal(out.view(word), bits)
