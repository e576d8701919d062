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
