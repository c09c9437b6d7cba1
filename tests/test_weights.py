"""Sums of attention weights without a GPU: refusals of the C interface and of the
binding, and the plain form that the GPU tests compare with."""

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
    (dict(q=None), 1), (dict(q=MIS), 1), (dict(lse=None), 1), (dict(kp=None), 1), (dict(ks=MIS), 1), (dict(sums=None), 1),
    (dict(sums=MIS), 1), (dict(lens=None), 1), (dict(bt=MIS), 1), (dict(Hq=3), 1), (dict(causal=2), 1),
    (dict(scale=0.0), 1), (dict(scale=1e-40), 1), (dict(scale=float("nan")), 1), (dict(decay=-0.5), 1),
    (dict(decay=float("inf")), 1), (dict(decay=float("nan")), 1), (dict(cu=A, Sn=4, max_q=0), 1),
    (dict(cu=A, Sn=4, max_q=5), 1), (dict(Hq=258), 2), (dict(D=96), 2), (dict(page=8), 2), (dict(B=1025), 2),
    (dict(B=1024, Sn=1 << 22), 2)])
def test_refusals(fa, kw, status):
    a = dict(q=A, lse=A, kp=A, ks=None, sums=A, B=2, Hq=4, Hkv=2, Sn=1, D=128, num_pages=8, page=16, max_pages=4, causal=1,
             scale=0.1, decay=1.0, bt=A, lens=A, cu=None, max_q=0)
    a.update(kw)
    assert fa.load_library().fa_cache_weights(*a.values(), None) == status


def test_binding_refuses_host_tensors(fa):
    x = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.cache_weights(x, torch.zeros(2, 2, 1), pages, torch.zeros(4, 2, 16), table, lens)


def test_plain_weights_add_up_to_the_rows():
    q, k = (np.random.default_rng(i).standard_normal((6, 4, 8)) for i in range(2))
    k = k[:, :2]
    for causal in (False, True):
        sees = P.causal_sees(4, 6, causal)
        lse = P.attention_of(q[:4], k, k, sees, 0.3)[1]
        w, slack = P.weights(q[:4], lse, k, sees, 0.3)
        assert np.allclose(w.sum(1), 8) and (slack >= 0).all()      # 4 tokens of 2 heads
        lse[1, 2] = -np.inf                                          # a row that gives nothing
        assert np.allclose(P.weights(q[:4], lse, k, sees, 0.3)[0].sum(1), [7, 8])
