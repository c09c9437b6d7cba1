"""Trees of drafted tokens without a GPU: refusals of the C interface and of the
binding, and the plain forms that the GPU tests compare with."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import paged as P

A = ctypes.c_void_p(1 << 20)          # never dereferenced
MIS = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


@pytest.mark.parametrize("kw,status", [
    (dict(parents=None), 1), (dict(mask=MIS), 1), (dict(depth=None), 1), (dict(cu=MIS, max_q=1), 1), (dict(B=0), 1),
    (dict(Sn=0), 1), (dict(cu=A, max_q=0), 1), (dict(cu=A, max_q=5), 1), (dict(Sn=1025), 2),
    (dict(cu=A, Sn=2000, max_q=1025), 2), (dict(B=1025), 2), (dict(cu=A, Sn=2 ** 31 - 1, max_q=4), 2)])
def test_mask_refusals(fa, kw, status):
    a = dict(parents=A, mask=A, depth=A, B=2, Sn=4, cu=None, max_q=0)
    a.update(kw)
    assert fa.load_library().fa_tree_mask(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(tree=None), 1), (dict(tree=MIS), 1), (dict(q=None), 1), (dict(Sn=1025), 2), (dict(ws=None), 5),
    (dict(cu=A, Sn=2000, max_q=1025), 2), (dict(cu=A, Sn=4, max_q=5), 1), (dict(D=96), 2), (dict(scale=0.0), 1)])
def test_attention_refusals(fa, kw, status):
    a = dict(q=A, kp=A, vp=A, ks=None, vs=None, o=A, lse=A, B=2, Hq=4, Hkv=2, Sn=3, D=128, num_pages=8, page=16,
             max_pages=4, tree=A, scale=0.1, bt=A, lens=A, cu=None, max_q=0, ws=A, nbytes=1 << 40)
    a.update(kw)
    assert fa.load_library().fa_fwd_paged_tree(*a.values(), None) == status


def test_binding_refuses_host_tensors(fa):
    with pytest.raises(ValueError):
        fa.tree_mask(torch.zeros(1, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        fa.tree_mask(torch.zeros(4, dtype=torch.int32), cu_seqlens=torch.zeros(2, dtype=torch.int32))


def test_plain_tree():
    sees, depth = P.tree_ancestors([-1, 0, 0, 1, -1, 4])
    assert depth.tolist() == [0, 1, 1, 2, 0, 1]
    assert [np.flatnonzero(r).tolist() for r in sees] == [[0], [0, 1], [0, 2], [0, 1, 3], [4], [4, 5]]
    assert P.pack_bits(sees, 1)[:, 0].tolist() == [1, 3, 5, 11, 16, 48]
    assert P.pack_bits(np.eye(34, dtype=bool), 2)[31].tolist() == [-2 ** 31, 0]
    full = P.tree_sees(sees, 8)          # two keys before the tree
    assert np.flatnonzero(full[3]).tolist() == [0, 1, 2, 3, 5]
    short = P.tree_sees(sees, 4)         # the first two tokens are padding
    assert not short[:2].any() and np.flatnonzero(short[3]).tolist() == [1] and np.flatnonzero(short[5]).tolist() == [2, 3]
    q, k, v = (np.random.default_rng(i).standard_normal((6, 1, 8)) for i in range(3))
    for causal in (False, True):         # the plain attention of a mask is the other one's
        a, b = P.attention(q, k, v, causal, 0.3), P.attention_of(q, k, v, P.causal_sees(6, 6, causal), 0.3)
        assert all(np.allclose(x, y, atol=1e-12) for x, y in zip(a, b))
