"""Trees whose tokens see few of the others, with nothing before the tree: rows whose first
blocks of keys, or whole shares of a split sequence, are masked throughout before one is
not."""

import numpy as np
import pytest
import torch

from oracle import paged as P

from paged_case import Cache, cu_of, randn
from tree_case import check_rows, words_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


def seen(n, kind):
    bits = np.zeros((n, n), dtype=bool)
    if kind == "itself":
        np.fill_diagonal(bits, True)
    elif kind == "last":
        bits[:, n - 1] = True
    elif kind == "first":
        bits[:, 0] = True
    else:                                   # some rows nothing, some one token, some the last block's
        bits[np.arange(0, n, 3), np.arange(0, n, 3)[::-1]] = True
        bits[1::3, n - n // 8 - 1:] = True
    return bits


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["itself", "last", "first", "mixed"])
@pytest.mark.parametrize("n,Hq,before", [(8, 2, 0), (16, 1, 100), (300, 4, 0), (700, 2, 0), (1024, 1, 5)])
def test_isolated_tokens(fa, n, Hq, before, kind, D, fp8):
    new, lens = [n, max(1, n // 3)], [n + before, max(1, n // 3)]
    c = Cache(lens, 1, D, 32, fp8, seed=n)
    bits = [seen(m, kind) for m in new]
    q = randn((sum(new), Hq, D), 3).cuda()
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, tree=words_of(bits, n, junk=True),
                          cu_seqlens=cu_of(new), max_q=n, **c.scales)
    assert fa.get_device_error() == 0
    check_rows(o, lse, q, c, new, [P.tree_sees(m, L) for m, L in zip(bits, lens)], D ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
def test_shares_without_a_key(fa, fp8):
    """One sequence over a long past whose tokens' own keys lie in the last share alone; and
    masks of nothing, whose rows see the past."""
    n, before = 600, 3000
    c = Cache([n + before, n], 1, 64, 128, fp8, seed=4)
    bits = [np.zeros((n, n), dtype=bool), seen(n, "last")]
    q = randn((2 * n, 2, 64), 3).cuda()
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, tree=words_of(bits, n), cu_seqlens=cu_of([n, n]),
                          max_q=n, **c.scales)
    assert fa.get_device_error() == 0
    check_rows(o, lse, q, c, [n, n], [P.tree_sees(m, L) for m, L in zip(bits, c.lens)], 0.125)
