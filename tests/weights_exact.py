"""Sums of weights whose scores are exact: queries and keys are small integers, so their
products' sums hold in FP32 in any order and however the tensor cores cut sums off.
What is left is what the formula itself rounds, and a score, or its difference to the
LSE, that is held in fewer bits shows."""

import numpy as np
import torch

from oracle import paged as P

from paged_case import Cache

SCALE = 2.0 ** -6


def integers(shape, most, seed):
    return np.random.default_rng(seed).integers(-most, most + 1, shape).astype(np.float64)


class IntegerCache(Cache):
    """Keys of whole numbers up to 8, which E4M3 rows hold exactly as well."""

    def __init__(self, lens, Hkv, D, page, fp8, seed=0, device="cuda"):
        super().__init__(lens, Hkv, D, page, fp8, seed=seed, device=device)
        rows = integers((sum(lens), Hkv, D), 8, seed)
        self.value["k"] = rows
        first = 0
        for b, n in enumerate(lens):
            t = np.arange(n)
            page_of, slot = torch.from_numpy(self.table[b, t // page]).long(), torch.from_numpy(t % page)
            own = rows[first:first + n]
            if fp8:
                codes, scale = P.quantise(own)
                assert np.array_equal(P.dequantise(codes, scale), own)
                self.host["k"][page_of, :, slot] = torch.from_numpy(codes)
                self.scale_host["k"][page_of, :, slot] = torch.from_numpy(scale)
            else:
                self.host["k"][page_of, :, slot] = torch.from_numpy(own).to(torch.bfloat16)
            first += n
        self.upload()


def queries(rows, Hq, D, seed):
    """Whole numbers up to 60: scores of some thousands, |sum| below 2^16."""
    return torch.from_numpy(integers((rows, Hq, D), 60, seed)).to(torch.bfloat16)


def expected(q, lse, k, sees, scale):
    """(sums [Hkv, L], what they may be off by) of one sequence; q [n, Hq, D], lse [Hq, n]
    (rows with -inf give nothing).  Of the score, exact, and the LSE, FP32, x is the
    difference, rounded once (2^-24 |x|) and once more in log2 units (2^-24 |x|, and
    2^-25 |x| for the constant); the exponential unit is good to 2^-22.  A sum of m
    weights is off by 2^-24 of itself for each, and weights below 2^-126 are zero."""
    n, Hq, _ = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    out, tol = np.zeros((Hkv, L)), np.zeros((Hkv, L))
    count = np.zeros((Hkv, L))
    for h in range(Hq):
        g = h // (Hq // Hkv)
        s = q[:, h] @ k[:, g].T * scale
        for i in range(n):
            if np.isneginf(lse[h, i]):
                continue
            x = np.where(sees[i], s[i] - lse[h, i], -np.inf)
            w = np.exp(x)
            out[g] += w
            tol[g] += np.where(sees[i], w * (2.5 * 2.0 ** -24 * np.abs(np.where(sees[i], x, 0)) + 2.0 ** -22), 0)
            count[g] += sees[i]
    return out, tol + (count + 1) * (2.0 ** -24 * out + 2.0 ** -125)


def logsumexp(q, k, sees, scale, alive):
    """FP32 LSE [Hq, n]; -inf where `alive` [Hq, n] is false."""
    n, Hq, _ = q.shape
    out = np.full((Hq, n), -np.inf)
    for h in range(Hq):
        s = np.where(sees, q[:, h] @ k[:, h // (Hq // k.shape[1])].T * scale, -np.inf)
        m = s.max(1)
        out[h] = m + np.log(np.exp(s - m[:, None]).sum(1))
    return np.where(alive, out, -np.inf).astype(np.float32)
