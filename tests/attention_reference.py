"""Plain 64-bit forms of the rollout's attention path for the tests: rotary
positions, the values of an NVFP4 paged cache, attention over them, and the
error bounds that follow from the library's number formats.  numpy on the CPU."""
import numpy as np

U32 = 2.0 ** -24  # half a step of fp32
BF16 = 2.0 ** -8  # half a step of bf16
FP16 = 2.0 ** -11


def rope(x, positions, inv_freq, interleaved, magnitude, inverse):
    """(y, bound): y in 64 bits; bound on an fp32 evaluation.  The half turns are
    rounded to fp32 (angle off by pi 2^-25), sine and cosine are within 2 steps,
    the magnitude and the two products round once each: under 8 U32 of
    m (|a| + |b|) together, the sum's rounding included."""
    x = x.astype(np.float64)
    h = len(inv_freq)
    a = positions.astype(np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(a) * magnitude, np.sin(a) * magnitude * (-1 if inverse else 1)
    y, bound = x.copy(), np.zeros_like(x)
    u = slice(0, 2 * h, 2) if interleaved else slice(0, h)
    w = slice(1, 2 * h, 2) if interleaved else slice(h, 2 * h)
    y[..., u] = x[..., u] * c - x[..., w] * s
    y[..., w] = x[..., u] * s + x[..., w] * c
    bound[..., u] = bound[..., w] = 8 * U32 * abs(magnitude) * (np.abs(x[..., u]) + np.abs(x[..., w]))
    return y, bound


def stored_values(codes, scales, st):
    """G s_b s_t of codes [..., D/2] and block scales [..., D/16] in 64 bits."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    g = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])[c & 7] * np.where(c & 8, -1.0, 1.0)
    e, m = ((scales >> 3) & 15).astype(np.float64), (scales & 7).astype(np.float64)
    sb = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7))
    return g * np.repeat(sb, 16, -1) * float(st)


def attention(q, keys, values, first, scale, causal, window):
    """One sequence: q [n, Hq, D] at positions first.., keys and values [L, Hkv,
    D], all 64-bit.  Returns (out, lse, tol): tol bounds an evaluation with
    exact products summed in fp32, an fp32 softmax, weights rounded to fp16 for
    the second product and a bf16 result.

    With A = sum p |v| (>= |out|): the weights' rounding moves out by FP16 A,
    a score error d moves it by 2 d A (numerator and sum).  d is the fp32 sum
    of D products, U32 D sum |q k| scale at most, plus a few roundings of the
    score itself (8 U32 |s| with the reference's subtraction and the base-2
    exponential).  The sums over the L keys add 2 L U32 A, and a rescaling or a
    joint a few more roundings.  FP16 is relative only for normal numbers: a
    weight under 2^-14 is rounded to a multiple of 2^-24, so it is off by 2^-25
    at most; the largest weight is at least 2^9 (the running reference is set 9
    below a new maximum and never lies nearer to it), so the sum of weights is
    too, and such a key moves out by 2^-34 |v|: 2^-34 sum |v| in all, which A
    does not cover where the keys of large weight have v = 0."""
    n, Hq, D = q.shape
    L, Hkv, _ = keys.shape
    g = Hq // Hkv
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    tol = np.zeros((n, Hq, D))
    j = np.arange(L)
    for i in range(n):
        see = (j <= first + i) if causal else np.ones(L, bool)
        if window > 0:
            see &= j > first + i - window
        if not see.any():
            continue
        for h in range(Hq):
            k, v = keys[see, h // g], values[see, h // g]
            s = k @ q[i, h] * scale
            top = s.max()
            p = np.exp(s - top)
            total = p.sum()
            p /= total
            lse[i, h] = top + np.log(total)
            out[i, h] = p @ v
            A = p @ np.abs(v)
            absum = (np.abs(k) @ np.abs(q[i, h])).max() * abs(scale)
            d = U32 * (D * absum + 8 * np.abs(s).max())
            tol[i, h] = BF16 * np.abs(out[i, h]) + A * (FP16 + 2 * d + 2 * len(s) * U32 + 64 * U32)
            tol[i, h] += 2.0 ** -34 * np.abs(v).sum(0)
    return out, lse, tol


class Pages:
    """A paged cache with random contents in host memory: the pages of each
    sequence in random order, every byte that no key owns set to 0xFF (block
    scales whose bit pattern is a NaN)."""

    def __init__(self, lens, Hkv, S, D, seed, share=(), spare=2, k_st=2.0 ** -6, v_st=0.0171):
        r = np.random.default_rng(seed)
        need = [-(-n // S) for n in lens]
        self.P, self.S, self.Hkv, self.D = sum(need) + spare, S, Hkv, D
        order = r.permutation(self.P)
        self.width = max([1, *need]) + 1
        self.table = np.full((len(lens), self.width), -7, np.int32)  # never read past a length
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        for b, other, m in share:  # sequence b's first m pages are another's
            self.table[b, :m] = self.table[other, :m]
        self.k_codes = np.full((self.P, Hkv, S, D // 2), 0xFF, np.uint8)
        self.v_codes = np.full((self.P, Hkv, S, D // 2), 0xFF, np.uint8)
        self.k_scales = np.full((self.P, Hkv, S, D // 16), 0xFF, np.uint8)
        self.v_scales = np.full((self.P, Hkv, D // 16, S), 0xFF, np.uint8)
        self.k_st, self.v_st = np.float32(k_st), np.float32(v_st)
        for b, n in enumerate(lens):
            for i in range(need[b]):
                m, pg = min(S, n - i * S), self.table[b, i]
                self.k_codes[pg, :, :m] = r.integers(0, 256, (Hkv, m, D // 2))
                self.v_codes[pg, :, :m] = r.integers(0, 256, (Hkv, m, D // 2))
                self.k_scales[pg, :, :m] = r.integers(0x20, 0x40, (Hkv, m, D // 16))
                self.v_scales[pg, :, :, :m] = r.integers(0x00, 0x70, (Hkv, D // 16, m))

    def rows(self, b, n):
        """(keys, values) [n, Hkv, D] of sequence b in 64 bits."""
        slots = np.arange(n)
        pg, off = self.table[b, slots // self.S], slots % self.S
        k = stored_values(self.k_codes[pg, :, off], self.k_scales[pg, :, off], self.k_st)
        v = stored_values(self.v_codes[pg, :, off], self.v_scales[pg, :, :, off], self.v_st)
        return k, v

    def cache(self, nvq):
        import torch

        t = [torch.from_numpy(a).cuda() for a in (self.k_codes, self.k_scales, self.v_codes, self.v_scales)]
        st = [torch.tensor([float(x)], dtype=torch.float32, device="cuda") for x in (self.k_st, self.v_st)]
        return nvq.KvCache(*t, *st)
