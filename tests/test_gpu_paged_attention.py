"""GPU parity of the attention over the paged NVFP4 cache with a 64-bit
evaluation: decoded tokens, drafts and prompt chunks, ragged and empty
sequences, pages that end inside a tile, windows, head layouts, strides."""
import numpy as np
import pytest

import attention_reference as ref
from helpers import log

pytestmark = pytest.mark.gpu


def _nvq():
    from qat_nvfp4_quantize_amd import nvq

    return nvq


def _batch(seqs, Hq, D, seed, gap=0, qs=1.0):
    """q bf16 [rows + gap, Hq, D] on the CPU, cu_q, kv_len of (new, length) pairs."""
    import torch

    g = torch.Generator().manual_seed(seed)
    n = sum(a for a, _ in seqs)
    q = (torch.randn(n + gap, Hq, D, generator=g) * qs).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum([a for a, _ in seqs])]).astype(np.int32)
    return q, cu, np.array([b for _, b in seqs], np.int32)


def _run(pages, seqs, Hq, causal=True, window=0, seed=1, gap=3, max_q="max", qs=1.0, scale=None, cache=None):
    """Runs the call with lse and checks every owned row against 64 bits and
    every other row for being left alone.  Returns (out, lse)."""
    import torch

    nvq = _nvq()
    D = pages.D
    q, cu, lens = _batch(seqs, Hq, D, seed, gap, qs)
    cache = cache or pages.cache(nvq)
    dev = dict(device="cuda")
    out = torch.full((len(q), Hq, D), 7.0, dtype=torch.bfloat16, **dev)
    lse = torch.full((len(q), Hq), 7.0, **dev)
    mq = max([1, *[a for a, _ in seqs]]) if max_q == "max" else max_q
    args = (torch.from_numpy(cu).cuda(), torch.from_numpy(lens).cuda(), torch.from_numpy(pages.table).cuda())
    nvq.nvq_paged_attention(q.cuda(), cache, *args, max_q=mq, causal=causal, window=window, lse=lse, out=out,
                            scale=scale)
    out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    qn = q.float().numpy().astype(np.float64)
    sc = D ** -0.5 if scale is None else scale
    for b, (n, length) in enumerate(seqs):
        k, v = pages.rows(b, length)
        want, wlse, tol = ref.attention(qn[cu[b]:cu[b + 1]], k, v, length - n, sc, causal, window)
        got = out[cu[b]:cu[b + 1]]
        off = np.abs(got - want)
        assert (off <= tol).all(), (b, n, length, float((off - tol).max()), float(np.abs(want).max()))
        gl = lse[cu[b]:cu[b + 1]]
        assert (np.isneginf(gl) == np.isneginf(wlse)).all(), (b, n, length)
        fin = np.isfinite(wlse)
        # the score error and the sum's, a few roundings of lse itself
        absum = (np.abs(qn[cu[b]:cu[b + 1]]).max(initial=0) * np.abs(k).sum(-1).max(initial=0)) * abs(sc)
        room = ref.U32 * (D * absum + 2 * length + 64 + 16 * np.abs(wlse[fin]).max(initial=0))
        assert (np.abs(gl[fin] - wlse[fin]) <= room).all(), (b, float(np.abs(gl[fin] - wlse[fin]).max()), room)
    assert (out[cu[-1]:] == 7.0).all() and (lse[cu[-1]:] == 7.0).all()
    return out, lse


def _wide(pages, keys=2048):
    """The same pages under a block table that covers at least so many keys."""
    pages.table = np.pad(pages.table, ((0, 0), (0, max(0, -(-keys // pages.S) - pages.width))), constant_values=-7)
    pages.width = pages.table.shape[1]
    return pages


# (new, length) of each sequence
DECODE = [(1, 1), (1, 37), (1, 640), (1, 16), (0, 50), (1, 129), (0, 0), (1, 300)]
DRAFTS = [(4, 4), (3, 200), (4, 65), (1, 33), (0, 9), (4, 517)]
CHUNKS = [(70, 70), (1, 300), (33, 190), (0, 12), (129, 260), (5, 5)]


@pytest.mark.parametrize("window", [0, 1, 60])
@pytest.mark.parametrize("D,Hq,Hkv,S", [(128, 8, 2, 16), (64, 6, 3, 32), (256, 4, 1, 64), (128, 3, 3, 128),
                                        (128, 16, 1, 16), (64, 40, 2, 16), (80, 5, 1, 16), (512, 2, 2, 32),
                                        (16, 4, 4, 16)])
@pytest.mark.parametrize("kind", ["decode", "drafts", "chunks"])
def test_attention_matches_64_bits(kind, D, Hq, Hkv, S, window):
    seqs = {"decode": DECODE, "drafts": DRAFTS, "chunks": CHUNKS}[kind]
    if kind == "chunks" and (Hq > 8 or D > 256):
        seqs = [(40, 70), (1, 90), (17, 17)]
    log(f"[attention] {kind} D={D} heads={Hq}/{Hkv} page={S} window={window}")
    pages = ref.Pages([b for _, b in seqs], Hkv, S, D, seed=D + Hq + S)
    _run(pages, seqs, Hq, window=window, seed=len(kind))


@pytest.mark.parametrize("D", [64, 128, 256, 48])
@pytest.mark.parametrize("seqs", [[(3, 100), (50, 64), (1, 1)], [(1, 90), (2, 33)]])
def test_attention_without_causal_mask(D, seqs):
    log(f"[attention] not causal D={D} {seqs}")
    _run(ref.Pages([b for _, b in seqs], 2, 16, D, seed=D), seqs, 4, causal=False)


@pytest.mark.parametrize("D", [128, 64, 256, 32])
@pytest.mark.parametrize("n", [3, 40])
def test_rows_before_the_first_key_are_empty(D, n):
    """More new tokens than keys: rows at negative positions see nothing."""
    log(f"[attention] empty rows D={D} n={n}")
    seqs = [(n, n - 2), (n, 0), (1, 0), (n, 1), (2, 200)]
    out, lse = _run(ref.Pages([b for _, b in seqs], 2, 16, D, seed=3), seqs, 4)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all()
    assert (out[n:2 * n + 1] == 0).all() and np.isneginf(lse[n:2 * n + 1]).all()


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 1), (64, 4, 2), (256, 6, 2)])
def test_long_contexts_split_over_workgroups(D, Hq, Hkv):
    log(f"[attention] long D={D}")
    seqs = [(1, 9001), (2, 5000), (0, 0), (1, 3)]
    _run(ref.Pages([b for _, b in seqs], Hkv, 64, D, seed=D), seqs, Hq)
    seqs = [(50, 4100), (1, 2050), (3, 1)]
    _run(ref.Pages([b for _, b in seqs], Hkv, 16, D, seed=D), seqs, Hq)
    _run(ref.Pages([b for _, b in seqs], Hkv, 16, D, seed=D), seqs, Hq, window=700)


def test_sharp_flat_and_large_scores():
    """Scores far apart (one key takes all), equal scores, scores of thousands."""
    seqs = [(2, 700), (1, 64), (90, 333)]
    for scale, qs in ((4.0, 3.0), (0.0, 1.0), (-0.5, 2.0), (1e-30, 1e30), (1e30, 1e-30)):
        log(f"[attention] scale={scale} q={qs}")
        for D in (128, 48):
            _run(ref.Pages([b for _, b in seqs], 2, 32, D, seed=5), seqs, 4, scale=scale, qs=qs)


def test_a_nan_stays_in_its_row():
    import torch

    nvq = _nvq()
    for D, n in ((128, 1), (128, 60), (48, 1), (256, 30)):
        seqs = [(n, 100), (n, 77)]
        pages = ref.Pages([b for _, b in seqs], 1, 16, D, seed=9)
        q, cu, lens = _batch(seqs, 4, D, 11)
        args = [torch.from_numpy(a).cuda() for a in (cu, lens, pages.table)]
        clean = nvq.nvq_paged_attention(q.cuda(), pages.cache(nvq), *args, max_q=n)
        q[0, 1, 5] = float("nan")
        q[n, 2, 3] = float("inf")
        dirty = nvq.nvq_paged_attention(q.cuda(), pages.cache(nvq), *args, max_q=n)
        assert torch.isnan(dirty[0, 1]).all()
        same = torch.ones(2 * n, 4, dtype=torch.bool, device="cuda")
        same[0, 1] = same[n, 2] = False
        assert torch.equal(dirty[same], clean[same]), (D, n)


def test_shared_pages_strides_and_head_major_queries():
    import torch

    nvq = _nvq()
    for D, seqs in ((128, [(1, 200), (1, 230), (2, 96)]), (128, [(40, 200), (64, 230), (2, 96)]),
                    (96, [(1, 60), (1, 80), (2, 40)])):
        pages = ref.Pages([b for _, b in seqs], 2, 16, D, seed=21, share=[(1, 0, 3), (2, 0, 2)])
        _run(pages, seqs, 8)
        q, cu, lens = _batch(seqs, 8, D, 1)
        args = [torch.from_numpy(a).cuda() for a in (cu, lens)]
        wide = torch.full((len(seqs), pages.width + 5), 2 ** 30, dtype=torch.int32)
        wide[:, 2:2 + pages.width] = torch.from_numpy(pages.table)
        table = wide.cuda()[:, 2:2 + pages.width]
        cache, dense = pages.cache(nvq), q.cuda()
        want = nvq.nvq_paged_attention(dense, cache, *args, torch.from_numpy(pages.table).cuda())
        fused = torch.randn(len(q), 13, D + 16, device="cuda").to(torch.bfloat16)
        fused[:, 2:10, :D] = dense
        out = torch.full((8, len(q), D), 3.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        got = nvq.nvq_paged_attention(fused[:, 2:10, :D], cache, *args, table, out=out)
        assert got is out and torch.equal(got, want), D
        again = nvq.nvq_paged_attention(dense.transpose(0, 1).contiguous().transpose(0, 1), cache, *args, table)
        assert torch.equal(again, want)


def test_bad_index_arrays_are_reported_and_stay_in_bounds():
    import torch

    nvq = _nvq()
    for D, n in ((128, 1), (128, 50), (64, 3), (48, 2)):
        seqs = [(n, 100), (n, 60), (n, 90)]
        pages = ref.Pages([b for _, b in seqs], 2, 16, D, seed=4)
        q, cu, lens = _batch(seqs, 4, D, 2)
        q, cache = q.cuda(), pages.cache(nvq)
        t = dict(dtype=torch.int32, device="cuda")

        def run(cu=cu, lens=lens, table=pages.table, max_q=n):
            cu, lens, table = (torch.as_tensor(np.asarray(a), **t) for a in (cu, lens, table))
            ws = nvq.workspace(64 << 20, "cuda")
            ws.fill_(0xFF)
            out = torch.full_like(q, 5.0)
            nvq.nvq_paged_attention(q, cache, cu, lens, table, max_q=max_q, ws=ws, out=out)
            return out, nvq.device_status(ws)

        clean, status = run()
        assert status == 0
        bad = pages.table.copy()
        bad[1, 1], bad[1, 3] = pages.P, -1
        out, status = run(table=bad)
        assert status == nvq.NVQ_STATUS_BAD_SEQUENCE
        assert torch.equal(out[:n], clean[:n]) and torch.equal(out[2 * n:], clean[2 * n:])
        qn = q[n:2 * n].float().cpu().numpy().astype(np.float64)  # such keys are left out
        k, v = pages.rows(1, 60)
        left = np.r_[0:16, 32:48]
        for i in range(n):
            see = left[left <= 60 - n + i]
            want, _, tol = ref.attention(qn[i:i + 1], k[see], v[see], 0, D ** -0.5, False, 0)
            assert (np.abs(out[n + i].float().cpu().numpy() - want[0]) <= tol[0]).all()
        out, status = run(lens=[100, -5, 90])
        assert status == nvq.NVQ_STATUS_BAD_SEQUENCE and not out[n:2 * n].any()
        assert torch.equal(out[2 * n:], clean[2 * n:])
        out, status = run(lens=[100, 2 ** 31 - 1, 90])
        assert status == nvq.NVQ_STATUS_BAD_SEQUENCE and torch.equal(out[2 * n:], clean[2 * n:])
        out, status = run(cu=[0, n, 2 * n, 2 ** 31 - 1])
        assert status == nvq.NVQ_STATUS_BAD_SEQUENCE and torch.equal(out[:2 * n], clean[:2 * n])
        out, status = run(cu=[-9, n, n - 1, 3 * n])
        assert status == nvq.NVQ_STATUS_BAD_SEQUENCE
        if n > 1:
            out, status = run(max_q=n - 1)
            assert status == nvq.NVQ_STATUS_BAD_SEQUENCE
            cut = torch.arange(3 * n, device="cuda") % n == n - 1
            assert (out[cut] == 5.0).all() and torch.equal(out[~cut], clean[~cut])
        # ids past the keys' pages are not looked at
        out, status = run()
        assert status == 0 and torch.equal(out, clean)


def test_nothing_to_do():
    import torch

    nvq = _nvq()
    pages = ref.Pages([5], 1, 16, 64, seed=1)
    cache = pages.cache(nvq)
    t = dict(dtype=torch.int32, device="cuda")
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(1, **t)
    assert nvq.nvq_paged_attention(none, cache, z, z[:0], torch.zeros(0, 0, **t)).shape == (0, 2, 64)
    q = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 4.0)
    nvq.nvq_paged_attention(q, cache, z, z[:0], torch.zeros(0, 4, **t), out=out)  # no sequence owns a row
    assert (out == 4.0).all()
    cu = torch.tensor([0, 3], **t)
    out = nvq.nvq_paged_attention(q, cache, cu, z, torch.zeros(1, 0, **t))  # a table without columns
    assert not out.any()


def test_pages_past_32_bits_of_bytes():
    import torch

    nvq = _nvq()
    Hkv, S, D = 8, 64, 128
    seqs = [(1, 300), (1, 90), (40, 200)]
    pages = ref.Pages([b for _, b in seqs], Hkv, S, D, seed=8)
    low = pages.cache(nvq)
    P = 2 ** 32 // (Hkv * S * D // 2) + pages.P + 5
    high = nvq.KvCache.empty(P, Hkv, S, D, 1.0, 1.0)
    for a, b in ((high.k_codes, low.k_codes), (high.k_scales, low.k_scales), (high.v_codes, low.v_codes),
                 (high.v_scales, low.v_scales), (high.k_scale, low.k_scale), (high.v_scale, low.v_scale)):
        a[-len(b):] = b
    for part in (seqs[:2], seqs):
        q, cu, lens = _batch(part, 16, D, 3)
        cu, lens = torch.from_numpy(cu).cuda(), torch.from_numpy(lens).cuda()
        table = torch.from_numpy(pages.table[:len(part)]).cuda()
        shifted = torch.where(table >= 0, table + (P - pages.P), table)
        n = max(a for a, _ in part)
        a = nvq.nvq_paged_attention(q.cuda(), low, cu, lens, table, max_q=n)
        b = nvq.nvq_paged_attention(q.cuda(), high, cu, lens, shifted, max_q=n)
        assert torch.equal(a, b)


@pytest.mark.parametrize("inter", [False, True])
def test_rollout_step_rotary_append_attend(inter):
    """The operators together, as a decoding layer uses them: projections in one
    fused tensor, queries and keys rotated in place, the new tokens appended,
    all tokens attending; a prompt chunk, then single tokens.  Each stage is
    compared with the 64-bit form of its own inputs."""
    import torch

    nvq = _nvq()
    B, Hq, Hkv, D, S = 3, 8, 2, 128, 16
    cache = nvq.KvCache.empty(40, Hkv, S, D, 42.0, 42.0)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(0xFF)
    g = torch.Generator().manual_seed(6)
    table = torch.randperm(40, generator=g)[:30].view(3, 10).to(torch.int32).cuda()
    f, m = nvq.nvq_rope_frequencies(D // 2, kind=nvq.NVQ_ROPE_RAMP, factor=4.0, orig_len=64.0)
    f = f.cuda()
    lens = np.zeros(B, np.int64)
    for new in ([40, 17, 100], [1, 1, 1], [1, 0, 1], [3, 2, 1]):
        new = np.array(new)
        T = int(new.sum())
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(lens, new)])
        owner = np.repeat(np.arange(B), new)
        lens = lens + new
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
        p = torch.from_numpy(pos.astype(np.int32)).cuda()
        o = torch.from_numpy(owner).cuda()
        slots = (table[o, (p // S).long()] * S + p % S).to(torch.int32)
        heads = qkv[:, :Hq + Hkv]
        x = heads.float().cpu().numpy()
        nvq.nvq_rope(heads, p, f, interleaved=inter, magnitude=m, out=heads)
        want, bound = ref.rope(x, pos, f.cpu().numpy(), inter, m, False)
        assert (np.abs(heads.float().cpu().numpy() - want) <= bound + ref.BF16 * np.abs(want)).all()
        k, v = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        nvq.nvq_kv_append(cache, k, v, slots)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        out = nvq.nvq_paged_attention(qkv[:, :Hq], cache, cu, ln, table, max_q=int(new.max()))
        q = qkv[:, :Hq].float().cpu().numpy().astype(np.float64)
        for b in range(B):
            every = torch.arange(int(lens[b]), device="cuda")
            sl = (table[b, every // S] * S + every % S).to(torch.int32)
            bk, bv = (t.double().cpu().numpy() for t in nvq.nvq_kv_gather(cache, sl, out_dtype=torch.float32))
            r = slice(int(cu[b]), int(cu[b + 1]))
            want, _, tol = ref.attention(q[r], bk, bv, int(lens[b] - new[b]), D ** -0.5, True, 0)
            # the fp32 read back is rounded where the call uses the exact product: U32 of each score and value
            assert (np.abs(out[r].float().cpu().numpy() - want) <= tol).all(), b


def test_captured_decode_step_replays_match_eager():
    """A decode step (rotary, append, attend) captured into a graph and replayed
    gives the eager step's bits, with the lengths, slots and positions advanced
    in place between replays and other eager calls on the same workspace."""
    import torch

    nvq = _nvq()
    B, Hq, Hkv, D, S = 5, 16, 2, 128, 32
    pages = ref.Pages([400, 31, 32, 90, 1], Hkv, S, D, seed=12)
    cache = pages.cache(nvq)
    t = dict(dtype=torch.int32, device="cuda")
    table = torch.from_numpy(pages.table).cuda()
    f = nvq.nvq_rope_frequencies(D)[0].cuda()
    cu = torch.arange(B + 1, **t)
    lens = torch.tensor([398, 29, 30, 88, 1], **t)
    qkv = torch.randn(B, Hq + 2 * Hkv, D, device="cuda").to(torch.bfloat16)
    pos, slots = torch.empty(B, **t), torch.empty(B, **t)
    ws = nvq.workspace(64 << 20, "cuda")
    seq = torch.arange(B, device="cuda")

    def advance(i):
        ln = torch.tensor([398 + i, 29 + i, 30 + i, 88 + i, 1], **t)
        lens.copy_(ln)
        pos.copy_(ln - 1)
        slots.copy_(table[seq, ((ln - 1) // S).long()] * S + (ln - 1) % S)

    def step():
        turned = nvq.nvq_rope(qkv[:, :Hq + Hkv], pos, f)
        nvq.nvq_kv_append(cache, turned[:, Hq:], qkv[:, Hq + Hkv:], slots, ws=ws)
        return nvq.nvq_paged_attention(turned[:, :Hq], cache, cu, lens, table, max_q=1, ws=ws)

    advance(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in (0, 1, 2, 1):
        advance(i)
        qkv.normal_()
        want = step().clone()
        ws.fill_(0x3C)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert nvq.device_status(ws) == 0


def test_side_stream_and_shared_workspace_of_two_shapes():
    import torch

    nvq = _nvq()
    seqs = [(1, 3000), (1, 40)]
    pages = ref.Pages([b for _, b in seqs], 2, 16, 128, seed=2)
    cache = pages.cache(nvq)
    q, cu, lens = _batch(seqs, 8, 128, 3)
    a = [torch.from_numpy(x).cuda() for x in (cu, lens, pages.table)]
    q = q.cuda()
    big = torch.randn(90, 8, 128, device="cuda").to(torch.bfloat16)
    cb = torch.tensor([0, 60, 90], dtype=torch.int32, device="cuda")
    want = nvq.nvq_paged_attention(q, cache, *a, max_q=1), nvq.nvq_paged_attention(big, cache, cb, *a[1:], max_q=60)
    torch.cuda.synchronize()
    ws = nvq.workspace(256 << 20, "cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            got = (nvq.nvq_paged_attention(q, cache, *a, max_q=1, ws=ws),
                   nvq.nvq_paged_attention(big, cache, cb, *a[1:], max_q=60, ws=ws))
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("D,Hq,Hkv,n", [(128, 16, 1, 3), (64, 12, 1, 5), (64, 33, 1, 1), (128, 71, 1, 1),
                                        (256, 16, 1, 2), (256, 17, 1, 2)])
def test_rows_of_every_kernel_variant(D, Hq, Hkv, n):
    """17 to 71 rows per key/value head: between the few-rows variants and past
    the last, beside single tokens and an empty sequence."""
    seqs = [(n, 333), (1, 130), (0, 0), (n, 5), (n, 2048)]
    for S in (16, 256):
        log(f"[attention] {n * Hq // Hkv} rows a head, D={D} page={S}")
        _run(ref.Pages([b for _, b in seqs], Hkv, S, D, seed=D + n), seqs, Hq)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seqs", [
    [(300, 300), (70, 1500)],              # several row tiles of 128 or 256
    [(40, 40 + 17 * i) for i in range(9)] + [(1, 600), (150, 150)],
    [(33, 5000), (200, 260)],              # few row tiles: their keys divided
    [(300, 2300), (90, 2100), (1, 70), (257, 257), (0, 9)],
    [(64, 64)] * 60,                       # many: handed out whole
])
def test_many_rows_divided_or_whole(D, seqs):
    log(f"[attention] D={D} {len(seqs)} sequences, first {seqs[:3]}")
    Hq = 4 if len(seqs) > 20 else 8
    pages = ref.Pages([b for _, b in seqs], 2, 64, D, seed=len(seqs))
    _run(pages, seqs, Hq)
    if len(seqs) < 20:
        _run(pages, seqs, Hq, window=130)
    if D == 128:  # 256-row tiles
        _run(_wide(pages), seqs, Hq)
        if len(seqs) < 20:
            _run(pages, seqs, Hq, window=1100)


@pytest.mark.parametrize("B,D,new,Hq,Hkv,far", [
    (70, 128, 1, 2, 1, 150), (300, 64, 2, 2, 1, 150), (1100, 64, 1, 2, 1, 150), (64, 128, 1, 32, 8, 1500),
    (200, 128, 2, 16, 16, 600), (100, 128, 5, 32, 8, 800), (90, 256, 2, 16, 8, 700), (100, 256, 9, 16, 8, 700),
    (120, 64, 5, 32, 16, 500), (100, 64, 20, 32, 16, 500), (70, 128, 16, 32, 8, 800)])
def test_many_sequences(B, D, new, Hq, Hkv, far):
    """More sequences than one step of the planning scans holds, empty ones among them."""
    log(f"[attention] {B} sequences D={D} {new} new tokens, heads {Hq}/{Hkv}")
    seqs = [(0 if i % 7 == 3 else new, (i * 37) % far + new) for i in range(B)]
    pages = ref.Pages([b for _, b in seqs], Hkv, 16, D, seed=B)
    _run(pages, seqs, Hq)
    _run(pages, seqs, Hq, window=33)
    if Hq > 2:
        return
    some = [(40 if i % 97 == 5 else n, max(b, 40)) for i, (n, b) in enumerate(seqs)]
    _run(ref.Pages([b for _, b in some], 1, 16, D, seed=B + 1), some, 2)


def test_pages_larger_than_a_tile():
    for S in (512, 4096):
        seqs = [(1, 5000), (70, 900), (3, 513), (130, 4097)]
        for D in (64, 128, 256):
            log(f"[attention] page={S} D={D}")
            _run(ref.Pages([b for _, b in seqs], 1, S, D, seed=S + D), seqs, 2)


@pytest.mark.parametrize("n,Hq", [(1, 4), (60, 4), (100, 8)])
@pytest.mark.parametrize("D", [64, 128, 256, 48])
@pytest.mark.parametrize("order", ["rising", "falling", "peak"])
def test_moving_reference(D, n, Hq, order):
    """Scores that climb by hundreds over the keys, so that the running
    reference moves and the sums are rescaled many times; that fall from the
    first key on; and one large score in the middle."""
    import torch

    length = 700
    log(f"[attention] {order} scores D={D} n={n}")
    pages = ref.Pages([length, length], 2, 16, D, seed=n + D)
    pages.k_codes &= 0x77  # magnitudes only: with positive queries all scores are positive
    for b in range(2):
        j = np.arange(length)
        climb = {"rising": j * 48 // length, "falling": 48 - j * 48 // length,
                 "peak": np.where(j == 333, 48, 4)}[order]
        pg, off = pages.table[b, j // 16], j % 16
        pages.k_scales[pg, :, off] = (0x10 + climb).astype(np.uint8)[:, None, None]
    nvq = _nvq()
    seqs = [(n, length), (n, length)]
    q, cu, lens = _batch(seqs, Hq, D, 5)
    q = q.abs()
    for scale, keys in ((2.0, 0), (30.0, 0), (2.0, 2048), (30.0, 2048)):
        args = [torch.from_numpy(x).cuda() for x in (cu, lens, _wide(pages, keys).table)]
        out = nvq.nvq_paged_attention(q.cuda(), pages.cache(nvq), *args, max_q=n, scale=scale)
        out = out.float().cpu().numpy().astype(np.float64)
        qn = q.float().numpy().astype(np.float64)
        for b in range(2):
            k, v = pages.rows(b, length)
            want, _, tol = ref.attention(qn[cu[b]:cu[b + 1]], k, v, length - n, scale, True, 0)
            assert (np.abs(out[cu[b]:cu[b + 1]] - want) <= tol).all(), (b, scale)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 63 - 1])
def test_windows_past_every_length(window):
    import torch

    nvq = _nvq()
    for D, seqs in ((128, [(3, 1), (2, 200)]), (128, [(60, 58), (2, 90)]), (48, [(3, 1), (2, 60)])):
        pages = ref.Pages([b for _, b in seqs], 1, 16, D, seed=3)
        q, cu, lens = _batch(seqs, 4, D, 8)
        args = [q.cuda(), pages.cache(nvq)] + [torch.from_numpy(x).cuda() for x in (cu, lens, pages.table)]
        a = nvq.nvq_paged_attention(*args)
        b = nvq.nvq_paged_attention(*args, window=window)
        assert torch.equal(a, b), (D, seqs)


def test_row_ranges_that_overlap_stay_in_bounds():
    """cu_q that falls and rises again: more row tiles than the rows make.  The
    buffers hold, the status word tells, rows of one owner are right."""
    import torch

    nvq = _nvq()
    n = 200
    seqs = [(n, 300)] * 5
    for D, Hq, keys in ((128, 4, 0), (128, 4, 2048), (64, 2, 0), (256, 2, 0), (48, 2, 0)):
        log(f"[attention] overlapping rows D={D}, table of {keys}")
        pages = _wide(ref.Pages([300] * 5, 1, 16, D, seed=D), keys)
        q = torch.randn(2 * n, Hq, D, device="cuda").to(torch.bfloat16)
        cache = pages.cache(nvq)
        lens = torch.full((5,), 300, dtype=torch.int32, device="cuda")
        table = torch.from_numpy(pages.table).cuda()

        def run(cu):
            ws = nvq.workspace(64 << 20, "cuda")
            out = torch.full_like(q, 5.0)
            cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
            nvq.nvq_paged_attention(q, cache, cu, lens, table, max_q=n, ws=ws, out=out)
            return out, nvq.device_status(ws)

        clean, status = run([0, n, n, n, n, 2 * n])
        assert status == 0
        out, status = run([n, 2 * n, 0, n, 0, n])
        assert status == nvq.NVQ_STATUS_BAD_SEQUENCE
        out, status = run([0, n, 0, n, 0, n])
        assert status == nvq.NVQ_STATUS_BAD_SEQUENCE and (out[n:] == 5.0).all()


def test_two_captured_graphs_share_a_workspace():
    """A prompt-chunk call and a decode call captured apart over one workspace,
    replayed in turn with eager calls on it between them."""
    import torch

    nvq = _nvq()
    seqs = [(90, 700), (40, 2100), (1, 33)]
    pages = ref.Pages([b for _, b in seqs], 2, 64, 128, seed=14)
    cache = pages.cache(nvq)
    lens, table = torch.tensor([700, 2100, 33], dtype=torch.int32).cuda(), torch.from_numpy(pages.table).cuda()
    big = torch.empty(131, 8, 128, dtype=torch.bfloat16, device="cuda")
    one = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    cb, co = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 90, 130, 131], [0, 1, 2, 3]))
    ws = nvq.workspace(256 << 20, "cuda")

    def chunk():
        return nvq.nvq_paged_attention(big, cache, cb, lens, table, max_q=90, ws=ws)

    def decode():
        return nvq.nvq_paged_attention(one, cache, co, lens, table, max_q=1, ws=ws)

    graphs, outs = [], []
    for f in (chunk, decode):
        big.normal_(), one.normal_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for i in range(4):
        big.normal_(), one.normal_()
        want = chunk().clone(), decode().clone()
        ws.fill_(0x7F if i % 2 else 0xFF)
        for k in ((0, 1), (1, 0), (0, 0), (1, 1))[i]:
            graphs[k].replay()
            if i % 2:
                torch.cuda.synchronize()
            assert torch.equal(outs[k], want[k]), (i, k)
        assert nvq.device_status(ws) == 0


def test_equal_calls_give_equal_bits():
    import torch

    nvq = _nvq()
    for seqs in ([(1, 4000), (1, 9), (1, 700)], [(80, 3000), (1, 500), (200, 900)]):
        pages = ref.Pages([b for _, b in seqs], 2, 16, 128, seed=6)
        q, cu, lens = _batch(seqs, 8, 128, 2)
        args = [q.cuda(), pages.cache(nvq)] + [torch.from_numpy(x).cuda() for x in (cu, lens, pages.table)]
        n = max(a for a, _ in seqs)
        first = nvq.nvq_paged_attention(*args, max_q=n)
        for _ in range(5):
            assert torch.equal(nvq.nvq_paged_attention(*args, max_q=n)[:cu[-1]], first[:cu[-1]])


@pytest.mark.parametrize("D,seqs", [(128, [(1, 3000), (1, 40), (2, 77)]), (256, [(1, 9)] * 70), (64, [(200, 5000)]),
                                    (128, [(300, 300), (1, 20), (70, 2500)]), (48, [(3, 50), (1, 9)])])
def test_output_in_place_of_the_queries(D, seqs):
    import torch

    nvq = _nvq()
    pages = ref.Pages([b for _, b in seqs], 2, 16, D, seed=D)
    q, cu, lens = _batch(seqs, 8, D, 4)
    q, args = q.cuda(), [pages.cache(nvq)] + [torch.from_numpy(x).cuda() for x in (cu, lens, pages.table)]
    n = max(a for a, _ in seqs)
    want = nvq.nvq_paged_attention(q, *args, max_q=n)
    got = nvq.nvq_paged_attention(q, *args, max_q=n, out=q)
    assert got is q and torch.equal(got, want)
