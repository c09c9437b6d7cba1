"""Sums of weights from exact scores: the kernels round what FP32 has to, and no more."""

import numpy as np
import pytest
import torch

from oracle import paged as P

from paged_case import cu_of
from parity import f64
from weights_exact import SCALE, IntegerCache, expected, logsumexp, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n,Hq,live", [(1, 4, 8), (4, 8, 20), (8, 8, 64), (9, 8, 2), (60, 8, 2), (60, 8, 960), (130, 6, 12)])
def test_exact_scores(fa, n, Hq, live, causal, D, fp8):
    """Two sequences of n tokens, `live` rows of theirs with an LSE."""
    lens, Hkv = [500, n + 37], 2
    c = IntegerCache(lens, Hkv, D, 32, fp8, seed=n + D)
    q = queries(2 * n, Hq, D, n)
    alive = np.zeros(2 * n * Hq, dtype=bool)
    alive[np.random.default_rng(2).permutation(2 * n * Hq)[:live]] = True
    alive = alive.reshape(Hq, 2 * n)
    sees = [P.causal_sees(n, L, causal) for L in lens]
    lse = np.concatenate([logsumexp(f64(q[b * n:(b + 1) * n]), c.rows("k", b), sees[b], SCALE, alive[:, b * n:(b + 1) * n])
                          for b in range(2)], 1)
    sums = torch.full(c.k_pages.shape[:3], float("nan"), device="cuda")
    fa.cache_weights(q.cuda(), torch.from_numpy(lse).cuda(), c.k_pages, sums, c.block_table, c.seq_lens, causal=causal,
                     scale=SCALE, decay=0.0, cu_seqlens=cu_of([n, n]), max_q=n, k_scale=c.k_scale)
    assert fa.get_device_error() == 0
    host = sums.cpu().numpy()
    for b, L in enumerate(lens):
        rows = slice(b * n, (b + 1) * n)
        want, tol = expected(f64(q[rows]), lse[:, rows].astype(np.float64), c.rows("k", b), sees[b], SCALE)
        t = np.arange(L)
        got = host[c.table[b, t // 32], :, t % 32].T.astype(np.float64)
        assert np.isfinite(got).all()
        assert np.all(np.abs(got - want) <= tol), (b, np.max(np.abs(got - want) / tol))
