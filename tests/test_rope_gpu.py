"""Rotary positions with several axes against the plain fp64 form.

Tolerance: a value is x cos - y sin in FP32, rounded once to BF16: 2^-8 of the
result, and 2^-20 of |x| + |y| for FP32 angles, sines and products."""

import numpy as np
import pytest
import torch

from oracle import paged as P

from paged_case import randn
from parity import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


def check(got, x, pos, sections, **kw):
    ref = P.rope(f64(x), pos, sections, kw.pop("base", 10000.0), **kw)
    mag = np.abs(P.rope(np.abs(f64(x)), pos * 0, sections, 10.0)).max(-1, keepdims=True)
    assert np.all(np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * mag)


@pytest.mark.parametrize("D,sections", [(128, [64]), (128, [16, 24, 24]), (64, [32]), (64, [8, 12, 12]), (128, [5, 3]),
                                        (64, [1]), (128, [24]), (64, [3, 5, 7, 2])])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("restart,inverse", [(False, False), (True, False), (False, True), (True, True)])
def test_rope(fa, D, sections, interleaved, restart, inverse):
    T, Hq, Hkv = 37, 6, 2
    q, k = randn((T, Hq, D), 1), randn((T, Hkv, D), 2)
    pos = np.random.default_rng(D + sum(sections)).integers(-50, 262144, (len(sections), T)).astype(np.int32)
    kw = dict(restart=restart, inverse=inverse, interleaved=interleaved)
    dpos = torch.from_numpy(pos).cuda()
    q2, k2 = fa.rope(q.cuda(), k.cuda(), dpos, sections=sections, **kw)
    check(q2, q, pos, sections, **kw)
    check(k2, k, pos, sections, **kw)
    # in place, and without keys: the same bits
    q3 = q.cuda()
    a, b = fa.rope(q3, None, dpos, sections=sections, q_out=q3, **kw)
    assert a is q3 and b is None and torch.equal(q3, q2)


@pytest.mark.parametrize("T", [1, 2, 607, 608, 1300, 5000])
def test_lengths(fa, T):
    q, k = randn((T, 3, 64), 1), randn((T, 1, 64), 2)
    pos = np.arange(T, dtype=np.int32)
    q2, k2 = fa.rope(q.cuda(), k.cuda(), torch.from_numpy(pos).cuda())
    check(q2, q, pos[None], [32])
    check(k2, k, pos[None], [32])


def test_dense_layout_and_base(fa):
    q, k = randn((2, 5, 4, 128), 1), randn((2, 5, 2, 128), 2)
    pos = np.random.default_rng(0).integers(0, 1000, (2, 2, 5)).astype(np.int32)
    q2, k2 = fa.rope(q.cuda(), k.cuda(), torch.from_numpy(pos).cuda(), sections=[32, 32], base=5e5)
    check(q2.view(10, 4, 128), q.view(10, 4, 128), pos.reshape(2, 10), [32, 32], base=5e5)
    check(k2.view(10, 2, 128), k.view(10, 2, 128), pos.reshape(2, 10), [32, 32], base=5e5)


def test_extreme_positions(fa):
    """The ends of int32: 2^31 positions of a turn's 2^-54 are 2^-22 turns."""
    pos = np.array([[-2 ** 31, 2 ** 31 - 1, -1, 0, 2 ** 27, -(2 ** 27)]], dtype=np.int32)
    q = randn((6, 1, 64), 1)
    q2, _ = fa.rope(q.cuda(), None, torch.from_numpy(pos).cuda())
    ref = P.rope(f64(q), pos, [32], 10000.0)
    assert np.all(np.abs(f64(q2) - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * np.pi * 2.0 ** -22 * 2 * np.abs(f64(q)).max())


def test_gradient_through_attention(fa):
    """Training: rope, fwd, bwd, and the inverse rotation of dQ and dK, against
    differences of a plain fp64 loss."""
    T, H, D, sections = 24, 1, 64, [10, 12, 10]
    q, k, v, do = (randn((1, T, H, D), s) for s in range(4))
    pos = np.random.default_rng(3).integers(0, 500, (3, T)).astype(np.int32)
    dpos = torch.from_numpy(pos).view(3, 1, T).cuda()
    q2, k2 = fa.rope(q.cuda(), k.cuda(), dpos, sections=sections)
    o, lse = fa.fwd(q2, k2, v.cuda(), causal=True)
    dq2, dk2, _ = fa.bwd(q2, k2, v.cuda(), o, lse, do.cuda(), causal=True)
    dq, dk = fa.rope(dq2, dk2, dpos, sections=sections, inverse=True)

    def loss(qx, kx):
        a, b = (P.rope(x, pos, sections, 10000.0) for x in (qx, kx))
        return (P.attention(a, b, f64(v)[0], True, D ** -0.5)[0] * f64(do)[0]).sum()

    qx, kx = f64(q)[0], f64(k)[0]
    rng = np.random.default_rng(5)
    for name, g in (("q", f64(dq)[0]), ("k", f64(dk)[0])):
        for _ in range(4):
            d = rng.normal(size=qx.shape)
            h = 1e-5
            args = [(qx + s * h * d, kx) if name == "q" else (qx, kx + s * h * d) for s in (1, -1)]
            diff = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            # the gradients are held to 1e-2 of their norm, rope's inputs and
            # outputs to 2^-8 each; a direction sees at most their norms' product
            tol = (1e-2 + 4 * 2.0 ** -8) * np.linalg.norm(g) * np.linalg.norm(d)
            assert abs((g * d).sum() - diff) <= tol
