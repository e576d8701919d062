"""GPU parity of the paged attention at the edges of its inputs: queries that
are not finite, tensor scales and queries far from one, single sequences of
every kernel variant and their mistakes in the index arrays."""
import numpy as np
import pytest

import attention_reference as ref
from helpers import log

pytestmark = pytest.mark.gpu

# batches that the few-rows kernel takes whole, divided and by single waves, the
# many-rows kernel and the kernel for any head dimension
# (head dimension, key/value heads, (new tokens, length) of each sequence)
KINDS = [(128, 1, [(1, 100), (2, 77)]), (64, 2, [(1, 9001), (2, 5000)]), (256, 1, [(2, 3000), (1, 40)]),
         (128, 16, [(2, 9 + 37 * i % 600) for i in range(100)]), (128, 1, [(90, 100), (70, 4000)]),
         (256, 2, [(50, 2100), (1, 9)]), (48, 1, [(1, 300), (3, 77)])]


def _nvq():
    from qat_nvfp4_quantize_amd import nvq

    return nvq


def _queries(seqs, Hq, D, seed, qs=1.0):
    """q bf16 [rows, Hq, D] on the CPU, and cu_q and kv_len of (new, length) pairs."""
    import torch

    n = sum(a for a, _ in seqs)
    q = (torch.randn(n, Hq, D, generator=torch.Generator().manual_seed(seed)) * qs).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum([a for a, _ in seqs])]).astype(np.int32)
    return q, cu, np.array([b for _, b in seqs], np.int32)


def _attend(pages, q, cu, lens, cache=None, ws=None, **more):
    """(out, lse) of one call, both on the GPU; rows and lse start as 7."""
    import torch

    nvq = _nvq()
    q = q.cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    args = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (cu, lens, pages.table)]
    more.setdefault("max_q", int(max(1, np.diff(cu).max())))
    nvq.nvq_paged_attention(q, cache or pages.cache(nvq), *args, lse=lse, out=out, ws=ws, **more)
    return out, lse


@pytest.mark.parametrize("D,Hkv,seqs", KINDS)
def test_log_sum_exp_of_a_query_that_is_not_finite(D, Hkv, seqs):
    """-inf stands for a row that sees no key: a NaN or infinite query has
    scores that are no numbers, and its lse must not be taken for that."""
    import torch

    log(f"[attention] lse of NaN and inf queries D={D} {len(seqs)} sequences, first {seqs[:2]}")
    pages = ref.Pages([b for _, b in seqs], Hkv, 16, D, seed=9)
    q, cu, lens = _queries(seqs, 2 * Hkv, D, 11)
    clean, clean_lse = _attend(pages, q, cu, lens)
    q[0, 1, 5] = float("nan")
    q[-1, 0, 3] = float("inf")
    out, lse = _attend(pages, q, cu, lens)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    assert not torch.isfinite(out[-1, 0]).any() and torch.isnan(lse[-1, 0])
    same = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    same[0, 1] = same[-1, 0] = False
    assert torch.equal(out[same], clean[same]) and torch.equal(lse[same], clean_lse[same])


def _compare(pages, seqs, q, cu, out, lse, scale, room=0.0):
    """Every row of (out, lse) against 64 bits.  room: what the result's format
    adds to the bound, where results are below its normal numbers."""
    out, lse = (t.double().cpu().numpy() for t in (out, lse))
    qn = q.double().numpy()
    for b, (n, length) in enumerate(seqs):
        k, v = pages.rows(b, length)
        r = slice(cu[b], cu[b + 1])
        want, wlse, tol = ref.attention(qn[r], k, v, length - n, scale, True, 0)
        off = np.abs(out[r] - want)
        assert (off <= tol + room).all(), (b, n, length, float((off - tol).max()), float(np.abs(want).max()))
        # the score error and the sum's, a few roundings of lse itself
        absum = np.abs(qn[r]).max(initial=0) * np.abs(k).sum(-1).max(initial=0) * abs(scale)
        near = ref.U32 * (pages.D * absum + 2 * length + 64 + 16 * np.abs(wlse).max(initial=0))
        assert (np.abs(lse[r] - wlse) <= near).all(), (b, n, length)


def _table_of(pages, keys):
    """Widens the block table to at least so many keys."""
    more = max(0, -(-keys // pages.S) - pages.width)
    pages.table = np.pad(pages.table, ((0, 0), (0, more)), constant_values=-7)
    pages.width += more


# Calls without a few-rows launch, whose many-rows launch looks the index arrays
# over itself: one sequence, or more than 64 query heads a key/value head.
# (D, query heads, key/value heads, sequences, keys of the table): the table's
# width chooses 256-row tiles at head dimension 128
ALONE = [(64, 8, 2, [(300, 900)], 0), (128, 8, 2, [(300, 900)], 0), (128, 8, 2, [(300, 900)], 2048),
         (128, 4, 1, [(150, 2600)], 0), (256, 8, 2, [(150, 900)], 0), (128, 70, 1, [(3, 300), (0, 9), (2, 77)], 0),
         (128, 70, 1, [(3, 300), (0, 9), (2, 77)], 2048), (256, 70, 1, [(3, 300), (2, 77)], 0)]


@pytest.mark.parametrize("D,Hq,Hkv,seqs,keys", ALONE)
def test_many_rows_alone(D, Hq, Hkv, seqs, keys):
    log(f"[attention] many rows alone D={D} heads={Hq}/{Hkv} {seqs} table of {keys}")
    pages = ref.Pages([b for _, b in seqs], Hkv, 64, D, seed=D + len(seqs))
    _table_of(pages, keys)
    q, cu, lens = _queries(seqs, Hq, D, 7)
    ws = _nvq().workspace(256 << 20, "cuda")
    out, lse = _attend(pages, q, cu, lens, ws=ws)
    assert _nvq().device_status(ws) == 0
    _compare(pages, seqs, q, cu, out, lse, D ** -0.5)


@pytest.mark.parametrize("D,Hq,Hkv,seqs,keys", ALONE)
def test_many_rows_alone_report_bad_index_arrays(D, Hq, Hkv, seqs, keys):
    import torch

    nvq = _nvq()
    log(f"[attention] bad index arrays, many rows alone D={D} heads={Hq}/{Hkv} {seqs} table of {keys}")
    pages = ref.Pages([b for _, b in seqs], Hkv, 64, D, seed=D)
    _table_of(pages, keys)
    q, cu, lens = _queries(seqs, Hq, D, 7)
    ws = nvq.workspace(256 << 20, "cuda")
    cache, table, last = pages.cache(nvq), pages.table, len(seqs) - 1

    def run(cu=cu, lens=lens, **more):
        out, lse = _attend(pages, q, cu, lens, cache, ws, **more)
        return out, lse, nvq.device_status(ws)

    def others_hold(out, lse):
        # Not bit by bit: one sequence's length moves the cuts through the others' keys, a part's reference is no
        # whole power of two, and so the weights under another reference round to other fp16 values.  Either
        # result is within the bound of the 64-bit one.
        _compare(pages, seqs[:last], q, cu, out, lse, D ** -0.5)

    def changed(a, at, value):
        a = a.copy()
        a[at] = value
        return a

    clean, _, status = run()
    assert status == 0
    bad = nvq.NVQ_STATUS_BAD_SEQUENCE
    for page in (pages.P, -1):
        pages.table = changed(table, (last, 1), page)
        out, lse, status = run()
        pages.table = table
        assert status == bad
        others_hold(out, lse)
    for length in (-5, 2 ** 31 - 1, pages.width * 64 + 1):
        out, lse, status = run(lens=changed(lens, last, length))
        assert status == bad
        others_hold(out, lse)
    n = int(np.diff(cu).max())
    for at, value in ((last + 1, cu[-1] + 1), (last + 1, 2 ** 31 - 1), (0, -1), (last + 1, cu[last] - 1)):
        assert run(cu=changed(cu, at, value), max_q=n)[2] == bad, (at, value)
    if n > 1:
        assert run(max_q=n - 1)[2] == bad
    out, _, status = run()
    assert status == 0 and torch.equal(out, clean)


def test_bad_pages_among_many_sequences_of_many_rows():
    """More sequences than one step of the check holds, in the 512-thread launch."""
    nvq = _nvq()
    seqs = [(2, 3 + i % 60) for i in range(600)]
    pages = ref.Pages([b for _, b in seqs], 1, 16, 128, seed=4)
    _table_of(pages, 2048)
    q, cu, lens = _queries(seqs, 70, 128, 7)
    ws = nvq.workspace(256 << 20, "cuda")
    cache, table = pages.cache(nvq), pages.table
    log("[attention] 600 sequences of 140 rows")
    _attend(pages, q, cu, lens, cache, ws)
    assert nvq.device_status(ws) == 0
    for b in (0, 255, 256, 599):
        log(f"[attention] bad page in sequence {b}")
        pages.table = table.copy()
        pages.table[b, 0] = pages.P
        _attend(pages, q, cu, lens, cache, ws)
        assert nvq.device_status(ws) == nvq.NVQ_STATUS_BAD_SEQUENCE, b


@pytest.mark.parametrize("v_st", [2.0 ** -126, 4e-40, 2.0 ** 112])
@pytest.mark.parametrize("D,Hkv,seqs", KINDS)
def test_tensor_scales_of_v_far_from_one(D, Hkv, seqs, v_st):
    """The sum of the weights may pass 2^26: divided by it, a small tensor scale
    is no normal number, though the output is.  Equal scores make the largest
    sums.  Outputs under 2^-126 are rounded to multiples of 2^-133 in bf16 (off
    by 2^-134), after an fp32 product that is off by 2^-150."""
    log(f"[attention] V scale {v_st} D={D} {len(seqs)} sequences, first {seqs[:2]}")
    pages = ref.Pages([b for _, b in seqs], Hkv, 16, D, seed=D, v_st=v_st)
    q, cu, lens = _queries(seqs, 2 * Hkv, D, 3)
    out, lse = _attend(pages, q, cu, lens, scale=0.0)
    _compare(pages, seqs, q, cu, out, lse, 0.0, 2.0 ** -134 + 2.0 ** -150)


@pytest.mark.parametrize("D,Hkv,seqs", KINDS + [(80, 1, [(40, 90), (1, 700)]), (512, 1, [(2, 40), (1, 70)])])
@pytest.mark.parametrize("power", [124, -124])
def test_queries_far_from_one(D, Hkv, seqs, power):
    """Finite queries near either end of bf16's range under a softmax scale that
    brings the scores back to a few units: no product on the way may leave fp32."""
    log(f"[attention] queries of 2^{power} D={D} {len(seqs)} sequences, first {seqs[:2]}")
    pages = ref.Pages([b for _, b in seqs], Hkv, 16, D, seed=D)
    q, cu, lens = _queries(seqs, 2 * Hkv, D, 5)
    q = q.clamp(-7.0, 7.0) * 2.0 ** power  # exact, below 2^127
    scale = 2.0 ** (2 - power) if power > 0 else 2.0 ** 126
    out, lse = _attend(pages, q, cu, lens, scale=scale)
    _compare(pages, seqs, q, cu, out, lse, scale)


def test_workspaces_with_gaps_are_refused_and_of_any_type_taken():
    """An expanded tensor has more elements than memory: it must not be written.
    A workspace of another type is as large as its bytes."""
    import torch

    nvq = _nvq()
    seqs = [(1, 3000), (2, 40)]
    pages = ref.Pages([b for _, b in seqs], 2, 16, 128, seed=2)
    q, cu, lens = _queries(seqs, 8, 128, 3)
    want, _ = _attend(pages, q, cu, lens)
    got, _ = _attend(pages, q, cu, lens, ws=torch.empty(4 << 20, dtype=torch.int64, device="cuda"))
    assert torch.equal(got, want)
    cache = pages.cache(nvq)
    x = torch.randn(3, 2, 128, device="cuda")
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    nvq.nvq_kv_append(cache, x, x, slots, ws=torch.empty(64, dtype=torch.int32, device="cuda"))
    for ws in (torch.empty(256, dtype=torch.uint8, device="cuda")[:1].expand(1 << 28),
               torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            _attend(pages, q, cu, lens, cache, ws)
        with pytest.raises(ValueError, match="contiguous"):
            nvq.nvq_kv_append(cache, x, x, slots, ws=ws)
        with pytest.raises(ValueError, match="contiguous"):
            nvq.nvq_kv_gather(cache, slots, ws=ws)
