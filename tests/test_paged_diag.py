"""Refusals of the paged attention with a wait limit of the caller's."""

import ctypes

import pytest

A = ctypes.c_void_p(1 << 20)          # never dereferenced


@pytest.mark.parametrize("limit,B,status", [(0, 2, 1), (10 ** 10 + 1, 2, 1), (10 ** 6, 0, 1), (10 ** 6, 1025, 2)])
def test_wait_limit_refusals(limit, B, status):
    import exact_attention_78_gb300 as fa
    lib = fa.load_library(build_if_missing=True)
    assert lib.fa_diag_fwd_paged(A, A, A, None, None, A, A, B, 4, 2, 1, 128, 8, 16, 4, 1, 0.1, A, A, None, 0, A, 1 << 40,
                                 limit, None) == status
