"""Refusals of rotary positions at the ends of what an int holds."""

import ctypes

import pytest

A = ctypes.c_void_p(1 << 20)          # never dereferenced


@pytest.mark.parametrize("tokens,status", [(2 ** 31 - 1, 2), (2 ** 31 - 512, 2), (-2 ** 31, 1)])
def test_token_counts(tokens, status):
    """Counts whose grid or last tokens would pass an int are refused ahead of the
    device."""
    import exact_attention_78_gb300 as fa
    lib = fa.load_library(build_if_missing=True)
    sections = (ctypes.c_int * 1)(32)
    assert lib.fa_rope(A, None, A, None, tokens, 1, 0, 64, A, 1, sections, 1e4, 0, 0, 0, None) == status
