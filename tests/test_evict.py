"""Eviction from a paged cache without a GPU: refusals of the C interface and of the
binding, and the plain selection that the GPU tests compare with."""

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
    (dict(sums=None), 1), (dict(sums=MIS), 1), (dict(index=None), 1), (dict(kept=MIS), 1), (dict(lens=None), 1),
    (dict(bt=None), 1), (dict(keep=0), 1), (dict(first=-1), 1), (dict(recent=-1), 1), (dict(keep=4, first=3, recent=2), 1),
    (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), 1), (dict(B=0), 1), (dict(page=48), 1), (dict(page=8), 2),
    (dict(B=1025), 2), (dict(Hkv=4097), 2), (dict(max_pages=1 << 27), 2), (dict(keep=2 ** 30 + 1), 2)])
def test_select_refusals(fa, kw, status):
    a = dict(sums=A, index=A, kept=A, B=2, Hkv=2, num_pages=8, page=16, max_pages=4, keep=8, first=1, recent=2, bt=A,
             lens=A)
    a.update(kw)
    assert fa.load_library().fa_cache_select(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(kp=None), 1), (dict(vp=MIS), 1), (dict(ks=A), 1), (dict(sums=MIS), 1), (dict(index=None), 1),
    (dict(counts=None), 1), (dict(counts=MIS), 1), (dict(start=MIS), 1), (dict(heads=2, Hkv=4), 1), (dict(heads=0), 1),
    (dict(most=0), 1), (dict(most=2 ** 30 + 1), 2), (dict(D=96), 2), (dict(page=8), 2), (dict(B=1025), 2), (dict(bt=MIS), 1)])
def test_keep_refusals(fa, kw, status):
    a = dict(kp=A, vp=A, ks=None, vs=None, sums=None, B=2, Hkv=2, D=128, num_pages=8, page=16, max_pages=4, bt=A, index=A,
             heads=2, most=8, counts=A, start=None)
    a.update(kw)
    assert fa.load_library().fa_cache_keep(*a.values(), None) == status


def test_binding_refuses_host_tensors(fa):
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.cache_select(torch.zeros(4, 2, 16), table, lens, 4)
    with pytest.raises(ValueError):
        fa.cache_keep(pages, pages, table, torch.zeros(2, 2, 4, dtype=torch.int32), lens)


def test_plain_selection():
    x = np.array([5.0, 1.0, 3.0, 3.0, 3.0, 0.0, 9.0, 0.5])
    assert P.select(x, 8, 0, 0).tolist() == list(range(8))
    assert P.select(x, 4, 0, 0).tolist() == [0, 2, 3, 6]
    assert P.select(x, 4, 2, 1).tolist() == [0, 1, 6, 7]
    assert P.select(x, 3, 0, 3).tolist() == [5, 6, 7]
    x[5], x[1] = np.nan, np.inf
    assert P.select(x, 1, 0, 0).tolist() == [5]
    assert P.select(x, 2, 0, 0).tolist() == [1, 5]
    assert P.select(np.array([-0.0, 0.0, -1.0]), 1, 0, 0).tolist() == [0]
