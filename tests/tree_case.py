"""Trees of drafted tokens over a small paged cache, with everything that a test
compares."""

import numpy as np
import torch

from oracle import paged as P

from paged_case import cu_of, randn
from parity import f64


def parents_of(n, seed, far=5):
    """A tree of n tokens: each follows one of the few before it, or none."""
    r = np.random.default_rng(seed)
    return np.array([max(-1, i - 1 - int(r.integers(0, far))) for i in range(n)], dtype=np.int32)


def masks(new, seed, kind="tree"):
    """Of each sequence, truth values [n, n]: a tree's, a chain's, random bits, or
    random bits with every third row empty."""
    out = []
    for b, n in enumerate(new):
        if kind == "tree":
            out.append(P.tree_ancestors(parents_of(n, seed + b))[0])
        elif kind == "chain":
            out.append(np.tril(np.ones((n, n), dtype=bool)))
        else:
            out.append(np.random.default_rng(seed + b).random((n, n)) < 0.3)
            if kind == "empty":
                out[-1][::3] = False
    return out


def words_of(bits, most, junk=False):
    """Masks as the library takes them, packed [total, W].  junk: the bits behind a tree's own are set."""
    W = -(-most // 32)
    rows = []
    for m in bits:
        full = np.full((m.shape[0], 32 * W), junk)
        full[:, :m.shape[1]] = m
        rows.append(P.pack_bits(full, W))
    return torch.from_numpy(np.concatenate(rows) if rows else np.zeros((0, W), dtype=np.int32)).cuda()


def check_rows(o, lse, q, c, new, sees, scale):
    """Packed O and LSE against the mask `sees` of each sequence.

    Tolerances as paged_case.check_attention's: O is rounded to BF16 (2^-8
    relative), so is each weight in the product and in the sum that it is divided by
    (2^-8 of sum |w v| / sum w, twice), 1e-5 for FP32 sums; a score is a sum of D
    products in FP32, off by at most D 2^-23 sum |q k| scale, and 2^-21 for
    exponentials and logarithm."""
    i = 0
    for b, n in enumerate(new):
        if n == 0:
            continue
        qb, k, v = f64(q[i:i + n]), c.rows("k", b), c.rows("v", b)
        o_ref, l_ref, a = P.attention_of(qb, k, v, sees[b], scale)
        ob, lb = f64(o[i:i + n]), f64(lse[:, i:i + n])
        assert np.isfinite(ob).all()
        np.testing.assert_array_equal(np.isfinite(lb), np.isfinite(l_ref))
        worst = np.max(np.abs(ob - o_ref) / (2.0 ** -8 * np.abs(o_ref) + 2.0 ** -7 * a + 1e-5))
        assert worst <= 1.0, (b, worst)
        assert not ob[np.isinf(l_ref).T].any()
        fin = np.isfinite(l_ref)
        if fin.any():
            span = np.abs(qb).sum(-1).max() * np.abs(k).max() * scale
            tol = q.shape[-1] * 2.0 ** -23 * span + 2.0 ** -21 * (1 + np.abs(l_ref[fin]).max())
            assert np.max(np.abs(lb[fin] - l_ref[fin])) <= tol
        i += n


def attend(fa, c, new, Hq, kind="tree", seed=3, dense=False, most=None, junk=False, **kw):
    """fwd_paged with trees, checked; returns packed (o, lse)."""
    most = max(new) if most is None else most
    bits = masks(new, seed, kind)
    tree = words_of(bits, most, junk)
    q = randn((sum(new), Hq, c.D), seed).cuda()
    scale = c.D ** -0.5
    args = (c.k_pages, c.v_pages, c.block_table, c.seq_lens)
    if dense:
        shape = (len(new), new[0])
        o, lse = fa.fwd_paged(q.view(*shape, Hq, c.D), *args, tree=tree.view(*shape, -1), **c.scales, **kw)
        o, lse = o.view(q.shape), lse.transpose(0, 1).reshape(Hq, -1)
    else:
        o, lse = fa.fwd_paged(q, *args, tree=tree, cu_seqlens=cu_of(new), max_q=most, **c.scales, **kw)
    assert fa.get_device_error() == 0
    check_rows(o, lse, q, c, new, [P.tree_sees(m, n) for m, n in zip(bits, c.lens)], scale)
    return o, lse
