"""Caches whose values show where each share of a row's weight went: column d of the
values is one for the d-th stretch of a sequence's keys and zero elsewhere, so O is
the weight that each stretch got.  With zero-mean values a lost or misplaced block
of a long sequence hides in the tolerance."""

import numpy as np
import torch

from oracle import paged as P

from paged_case import Cache
from parity import f64


def one_hot_values(length, Hkv, D):
    """[length, Hkv, D]: key t counts in column t // ceil(length / D), turned on by
    one column from head to head."""
    v = np.zeros((length, Hkv, D))
    t = np.arange(length)
    for h in range(Hkv):
        v[t, h, (t // -(-length // D) + h) % D] = 1.0
    return v


def shares_cache(lens, Hkv, D, page, fp8, seed=0, device="cuda"):
    c = Cache(lens, Hkv, D, page, fp8, seed=seed, device=device)
    v = np.concatenate([one_hot_values(n, Hkv, D) for n in lens])
    c.value["v"] = v
    codes, scale = P.quantise(np.eye(1, D)) if fp8 else (None, None)
    first = 0
    for b, n in enumerate(lens):
        for t in range(n):
            p, s = P.slot_of(c.table, page, b, t)
            if fp8:        # a row's one is the same code, at the same scale
                c.host["v"][p, :, s] = torch.from_numpy((v[first + t] * float(codes[0, 0])).astype(np.uint8))
                c.scale_host["v"][p, :, s] = int(scale[0])
            else:
                c.host["v"][p, :, s] = torch.from_numpy(v[first + t]).to(torch.bfloat16)
        first += n
    c.upload()
    return c


def tolerance(o_ref, a, q, k, scale, fp8):
    """What O may be off by, |w v| / sum w being `a`.  O is rounded to BF16, half a
    step, 2^-8 of it.  BF16 pages: each weight is rounded to BF16, 2^-8 of it, in
    the product and in the sum that divides.  E4M3: to FP16, 2^-11 of it, and no
    less than 2^-31 of the largest, in the product alone.  FP32: a score is a sum
    of D products (D 2^-23 of the sum of their sizes), which a weight follows, in
    the product and in the sum; a sum over keys goes 16 at a time; 2^-20 for
    exponentials and joining."""
    D, L = k.shape[-1], k.shape[0]
    span = np.abs(q).sum(-1).max() * np.abs(k).max() * scale
    fp32 = 2 * D * 2.0 ** -23 * span + 2 * (L / 16) * 2.0 ** -23 + 2.0 ** -20
    held = (2.0 ** -11, L * 2.0 ** -31) if fp8 else (2.0 ** -7, 0.0)
    return 2.0 ** -8 * np.abs(o_ref) + (held[0] + fp32) * a + held[1] + 2.0 ** -40


def worst(o, q, k, v, causal, scale, fp8):
    """The largest error of one sequence's O over its tolerance."""
    o_ref, _, a = P.attention(q, k, v, causal, scale)
    return np.max(np.abs(o - o_ref) / tolerance(o_ref, a, q, k, scale, fp8))


def check_shares(o, q, cache, new, causal, scale):
    first = 0
    for b, n in enumerate(new):
        if n:
            rows = slice(first, first + n)
            w = worst(f64(o[rows]), f64(q[rows]), cache.rows("k", b), cache.rows("v", b), causal, scale, cache.fp8)
            assert w <= 1.0, (b, w)
        first += n
