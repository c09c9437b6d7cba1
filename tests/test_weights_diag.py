"""Refusals of cache_weights with a wait limit of the caller's, and what the source of its
kernel of few rows says about waiting, without a GPU."""

import ctypes
import os
import re

import pytest

from test_bounded_waits import CSRC, functions

A = ctypes.c_void_p(1 << 20)          # never dereferenced


@pytest.mark.parametrize("limit,held,D,B,status", [
    (0, -1, 128, 2, 1), (10 ** 10 + 1, -1, 128, 2, 1), (10 ** 6, -2, 128, 2, 1), (10 ** 6, 18, 128, 2, 1),
    (10 ** 6, 22, 64, 2, 1), (10 ** 6, 17, 128, 0, 1), (10 ** 6, 21, 64, 1025, 2)])
def test_refusals(limit, held, D, B, status):
    import exact_attention_78_gb300 as fa
    lib = fa.load_library(build_if_missing=True)
    assert lib.fa_diag_cache_weights(A, A, A, None, A, B, 4, 2, 1, D, 8, 16, 4, 1, 0.1, 1.0, A, A, None, 0, limit, held,
                                     None) == status


def test_few_rows_wait_with_a_bound():
    """Each warp is on its own after the tables: no barrier of the block's that a warp which
    gave up would not come to, and no wait without a limit or an answer."""
    with open(os.path.join(CSRC, "fa_weights.cu")) as f:
        text = f.read()
    found = functions(text[text.index("step_kernel(const WeighParams p)"):])["step_kernel"]
    loop = found[found.index("while (at.left > 0)"):]
    assert loop.count("wait_warp(") == 1 and "p.wait_limit_ns" in loop
    assert not re.search(r"__syncthreads|bar\.sync|barrier\.sync|mbar_try_wait|mbar_wait\(", loop)
    assert not re.search(r"^\s*paged::wait_warp\(", loop, flags=re.M)
