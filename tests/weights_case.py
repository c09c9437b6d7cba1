"""Sums of attention weights over a small paged cache, checked against fp64."""

import numpy as np
import torch

from oracle import paged as P

from paged_case import cu_of, randn
from parity import f64


def lse_of(q, c, new, causal, scale):
    """FP32 LSE of packed rows, [Hq, total], by the plain form."""
    out, i = np.full((q.shape[1], q.shape[0]), np.nan, dtype=np.float32), 0
    for b, n in enumerate(new):
        if n:
            k = c.rows("k", b)
            out[:, i:i + n] = P.attention_of(f64(q[i:i + n]), k, k, P.causal_sees(n, c.lens[b], causal), scale)[1]
        i += n
    return torch.from_numpy(out)


def old_sums(c, seed, fill=float("nan")):
    """Sums of all tokens, `fill` in the slots that are no token's and in those of
    the new tokens' (which start anew)."""
    shape = tuple(c.k_pages.shape[:3])
    host = np.full(shape, fill, dtype=np.float32)
    r = np.random.default_rng(seed)
    for b, L in enumerate(c.lens):
        t = np.arange(L)
        host[c.table[b, t // c.page], :, t % c.page] = r.random((L, shape[1])) * 3
    return host


def check(fa, c, new, Hq, causal=True, decay=1.0, seed=3, dense=False, scale=None, q=None, lse=None, max_q=None, tail=0,
          stream=None):
    """cache_weights on cache c; every slot is compared.

    Tolerances.  A score is a sum of D products in FP32, off by at most
    D 2^-23 sum |q k| scale; its difference x to the LSE and that in log2 units are
    rounded to 2^-24 each, and the exponential is good to 2^-22: a weight is off by
    (D 2^-23 span + 2^-23 |x| + 2^-21) of itself.  A sum of m terms adds m 2^-24, decay
    and the old sum 2^-23."""
    total = sum(new)
    q = randn((total + tail, Hq, c.D), seed) if q is None else q
    scale = c.D ** -0.5 if scale is None else scale
    lse = lse_of(q[:total], c, new, causal, scale) if lse is None else lse
    full = torch.full((Hq, total + tail), float("nan"))
    full[:, :total] = lse
    before = old_sums(c, seed)
    i = 0
    for b, n in enumerate(new):
        t = np.arange(max(0, c.lens[b] - n), c.lens[b])
        before[c.table[b, t // c.page], :, t % c.page] = np.nan
    sums = torch.from_numpy(before).cuda()
    args = (c.k_pages, sums, c.block_table, c.seq_lens)
    kw = dict(causal=causal, decay=decay, scale=scale, k_scale=c.k_scale, stream=stream)
    if dense:
        B, n = len(new), new[0]
        fa.cache_weights(q.cuda().view(B, n, Hq, c.D), lse.view(Hq, B, n).transpose(0, 1).contiguous().cuda(), *args, **kw)
    else:
        fa.cache_weights(q.cuda(), full.cuda(), *args, cu_seqlens=cu_of(new), max_q=max_q or max(new), **kw)
    assert fa.get_device_error() == 0
    after = sums.cpu().numpy()
    same = np.ones(before.shape, dtype=bool)
    for b, n in enumerate(new):
        L = c.lens[b]
        if n == 0 or L == 0:
            i += n
            continue
        t = np.arange(L)
        at = (c.table[b, t // c.page], slice(None), t % c.page)
        qb, k = f64(q[i:i + n]), c.rows("k", b)
        want, slack = P.weights(qb, lse[:, i:i + n].numpy().astype(np.float64), k, P.causal_sees(n, L, causal), scale)
        old = before[at].astype(np.float64).T * float(np.float32(decay))       # (an FP32 argument)
        old[:, max(0, L - n):] = 0
        if decay == 0:
            old[:] = 0
        span = np.abs(qb).sum(-1).max() * np.abs(k).max() * scale
        rel = c.D * 2.0 ** -23 * span + 2.0 ** -21 + n * (Hq // c.Hkv) * 2.0 ** -24
        tol = want * rel + slack * 2.0 ** -23 + 2.0 ** -23 * (old + want) + 1e-30
        got = after[at].T
        assert np.isfinite(got).all()
        worst = np.max(np.abs(got - want - old) / tol)
        assert worst <= 1.0, (b, worst)
        same[at] = False
        i += n
    np.testing.assert_array_equal(after[same], before[same])
    return after
