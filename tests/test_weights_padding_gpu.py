"""Sums of attention weights of a padded batch: its padding gives no weight and may hold
anything."""

import numpy as np
import pytest
import torch

from paged_case import Cache, randn
from weights_case import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,Hq", [(3, 4), (30, 1), (40, 4), (90, 6)])
def test_padded_batch(fa, n, Hq, fp8):
    """Sequences with fewer keys than tokens, one without keys, one longer; queries and LSE of
    the padding are NaN, as memory that nobody wrote may be."""
    lens = [n - 2, n, 1, 0, n + 50]
    c = Cache(lens, 1, 128, 16, fp8, seed=n)
    q = randn((len(lens), n, Hq, 128), 2).cuda()
    _, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, **c.scales)
    good = torch.zeros(c.k_pages.shape[:3], device="cuda")
    fa.cache_weights(q, lse, c.k_pages, good, c.block_table, c.seq_lens, k_scale=c.k_scale)
    flat, rows = q.view(-1, Hq, 128).cpu(), lse.transpose(0, 1).reshape(Hq, -1).cpu()
    check(fa, c, [n] * len(lens), Hq, q=flat, lse=rows, dense=True)
    for b, L in enumerate(lens):
        q[b, :max(0, n - L)] = float("nan")
        lse[b, :, :max(0, n - L)] = float("nan")
    got = torch.zeros_like(good)
    fa.cache_weights(q, lse, c.k_pages, got, c.block_table, c.seq_lens, k_scale=c.k_scale)
    assert fa.get_device_error() == 0
    assert torch.equal(got, good)
    assert int(torch.isfinite(got).all()) and int(got.count_nonzero()) <= sum(lens)
