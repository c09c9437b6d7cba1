"""Sums of attention weights where the new tokens were a tree of drafts: once the accepted
ones lie together, each of them saw what the causal mask gives, so their rows of the
tree's q and LSE are what cache_weights takes."""

from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import paged as P

from paged_case import Cache, cu_of, randn
from parity import f64
from tree_case import parents_of
from weights_case import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


def ints(x):
    return torch.tensor(np.array(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq,decay", [(6, 4, 1.0), (40, 8, 0.75), (90, 6, 1.0)])
def test_accepted_drafts(fa, n, Hq, decay, D, fp8):
    Hkv, page = 2, 16
    past = [100, 17, 64, 0, 33]
    B = len(past)
    c = Cache([L + n for L in past], Hkv, D, page, fp8, seed=n)      # the drafts' keys are there
    parents = [parents_of(n, 5 + b, far=3) for b in range(B)]
    q = randn((B, n, Hq, D), 4).cuda()
    mask, _ = fa.tree_mask(ints(parents))
    _, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, tree=mask, **c.scales)

    # the ancestors of some token; of the last sequence none
    sees = [P.tree_ancestors(p)[0] for p in parents]
    paths = [np.flatnonzero(sees[b][n - 1 - b]) for b in range(B - 1)] + [np.zeros(0, dtype=int)]
    counts = [len(p) for p in paths]
    index = np.full((B, 1, max(counts)), -1, dtype=np.int32)
    for b, p in enumerate(paths):
        index[b, 0, :len(p)] = past[b] + p
    fa.cache_keep(c.k_pages, c.v_pages, c.block_table, ints(index), ints(counts), ints(past), **c.scales)
    assert fa.get_device_error() == 0

    lens = [L + m for L, m in zip(past, counts)]
    rows = [np.concatenate([c.rows("k", b)[:past[b]], c.rows("k", b)[past[b] + p]]) for b, p in enumerate(paths)]
    for b, p in enumerate(paths):                                    # what the tree's masks let them see
        of_tree = P.tree_sees(sees[b], past[b] + n)[p][:, np.concatenate([np.arange(past[b]), past[b] + p])]
        np.testing.assert_array_equal(of_tree, P.causal_sees(counts[b], lens[b], True))
    kept = SimpleNamespace(lens=lens, rows=lambda name, b: rows[b], table=c.table, page=page, D=D, Hkv=Hkv, k_pages=c.k_pages,
                           k_scale=c.k_scale, block_table=c.block_table, seq_lens=ints(lens))
    at = torch.cat([torch.from_numpy(b * n + p) for b, p in enumerate(paths)]).cuda()
    q_rows = q.view(B * n, Hq, D)[at]
    lse_rows = lse.transpose(0, 1).reshape(Hq, B * n)[:, at].contiguous()
    sums = check(fa, kept, counts, Hq, decay=decay, q=q_rows.cpu(), lse=lse_rows.cpu())

    # every row's weights add up to one (the LSE and the weights are off by 2^-18 or so each)
    fresh = torch.zeros(c.k_pages.shape[:3], device="cuda")
    fa.cache_weights(q_rows, lse_rows, c.k_pages, fresh, c.block_table, ints(lens), cu_seqlens=cu_of(counts),
                     max_q=max(counts), k_scale=c.k_scale)
    np.testing.assert_allclose(fresh.double().sum((0, 2)).cpu().numpy(), [sum(counts) * Hq // Hkv] * Hkv, rtol=1e-4)

    # and the sums choose what a head keeps
    dev = torch.from_numpy(sums).cuda()
    got, left = fa.cache_select(dev, c.block_table, ints(lens), 40, first=2, recent=5)
    assert fa.get_device_error() == 0 and left.tolist() == [min(L, 40) for L in lens]
    for b, L in enumerate(lens):
        t = np.arange(L)
        for h in range(Hkv):
            want = P.select(sums[c.table[b, t // page], h, t % page], 40, 2, 5)
            np.testing.assert_array_equal(got[b, h, :len(want)].cpu().numpy(), want)
