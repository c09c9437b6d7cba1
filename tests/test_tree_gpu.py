"""Trees of drafted tokens: their masks, and attention over a paged cache with
them, against plain fp64 forms."""

import numpy as np
import pytest
import torch

from oracle import paged as P

from paged_case import Cache, cu_of, randn
from tree_case import attend, masks, parents_of, words_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


def check_masks(parents, new, most, mask, depth):
    i = 0
    for b, n in enumerate(new):
        if n == 0:
            continue
        sees, d = P.tree_ancestors(parents[b])
        np.testing.assert_array_equal(mask[i:i + n].cpu().numpy(), P.pack_bits(sees, -(-most // 32)))
        np.testing.assert_array_equal(depth[i:i + n].cpu().numpy(), d)
        i += n


@pytest.mark.parametrize("new,most", [([1], 1), ([31, 32, 33], 33), ([5, 0, 64, 1], 100), ([1024, 3, 600], 1024)])
def test_masks_packed(fa, new, most):
    parents = [parents_of(n, b, far=1 if b == 2 else 40) for b, n in enumerate(new)]      # (far = 1: a chain)
    total = sum(new) + 3
    flat = torch.full((total,), 99, dtype=torch.int32)
    flat[:sum(new)] = torch.from_numpy(np.concatenate(parents))
    mask = torch.full((total, -(-min(most, total) // 32)), 7, dtype=torch.int32, device="cuda")
    depth = torch.full((total,), 7, dtype=torch.int32, device="cuda")
    fa.tree_mask(flat.cuda(), cu_of(new), max_q=min(most, total), mask=mask, depth=depth)
    assert fa.get_device_error() == 0
    check_masks(parents, new, min(most, total), mask, depth)
    assert (mask[sum(new):] == 7).all() and (depth[sum(new):] == 7).all()      # behind the last tree


def test_masks_dense_and_default_bound(fa):
    parents = [parents_of(45, b, far=9) for b in range(70)]
    flat = torch.from_numpy(np.stack(parents)).cuda()
    mask, depth = fa.tree_mask(flat)
    assert mask.shape == (70, 45, 2) and depth.shape == (70, 45)
    check_masks(parents, [45] * 70, 45, mask.view(-1, 2), depth.view(-1))
    mask, depth = fa.tree_mask(flat[0].contiguous(), cu_of([45]))
    check_masks(parents[:1], [45], 45, mask, depth)
    assert fa.get_device_error() == 0


def test_masks_of_bad_input(fa):
    p = torch.tensor([[-1, 0, 2, 7, -2, 1]], dtype=torch.int32, device="cuda")
    mask, depth = fa.tree_mask(p)
    assert fa.get_device_error() == 1
    check_masks([[-1, 0, -1, -1, -1, 1]], [6], 6, mask[0], depth[0])
    ok = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    for cu in ([0, 4, 3], [1, 2, 6], [0, 2, 7], [0, 6, 6], [-1, 2, 6]):
        out = torch.full((6, 1), 7, dtype=torch.int32, device="cuda")
        fa.tree_mask(ok, torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q=5, mask=out)
        assert fa.get_device_error() == 1, cu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 128, 1024])
@pytest.mark.parametrize("n,Hq,Hkv", [(1, 4, 2), (7, 2, 2), (4, 8, 2), (16, 2, 2), (32, 1, 1), (33, 4, 2), (100, 4, 1)])
def test_trees(fa, n, Hq, Hkv, page, D, fp8):
    """From the decode kernel's single tiles to several tiles of the chunk kernel."""
    c = Cache([n, n + 1, n + 15, n + 130, 300 + n], Hkv, D, page, fp8, seed=n + page)
    attend(fa, c, [n] * 5, Hq, dense=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["tree", "bits"])
@pytest.mark.parametrize("new,lens,Hq", [([3, 0, 8, 1], [70, 5, 8, 200], 2), ([60, 0, 200, 1], [700, 5, 200, 129], 8)])
def test_ragged(fa, new, lens, Hq, kind, D, fp8):
    """Any bits will do; those behind a tree's own mean nothing."""
    c = Cache(lens, 2, D, 32, fp8, seed=D)
    attend(fa, c, new, Hq, kind=kind, junk=True, most=max(new) + 1)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,Hq", [([8, 3, 8], 2), ([60, 200, 129], 8)])
def test_empty_rows(fa, new, Hq, fp8):
    """Tokens that see none of the tree, and no key at all where none lies before it."""
    c = Cache([new[0], new[1] + 40, new[2] - 2], 2, 64, 32, fp8, seed=4)
    o, lse = attend(fa, c, new, Hq, kind="empty")
    assert torch.isinf(lse[:, 0]).all() and not o[0].any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,Hq", [(8, 1), (90, 4)])
def test_padded_trees(fa, n, Hq, fp8):
    """Sequences with fewer keys than tokens: the first tokens are padding."""
    c = Cache([n - 3, n, 1, 0, n + 40], 1, 128, 16, fp8, seed=n)
    attend(fa, c, [n] * 5, Hq, dense=True)
    attend(fa, c, [n] * 5, Hq, kind="bits", dense=True)


@pytest.mark.parametrize("D", [64, 128])
def test_largest_tree(fa, D):
    c = Cache([1024 + 77, 1024], 1, D, 64, False, seed=2)
    attend(fa, c, [1024, 1000], 2)


def test_long_past_is_split(fa):
    """One sequence, whose keys all thread blocks share, its tree at the end."""
    for n, fp8 in ((2, False), (40, False), (40, True)):
        c = Cache([9000 + n], 1, 128, 128, fp8, seed=8)
        attend(fa, c, [n], 8)


@pytest.mark.parametrize("fp8", [False, True])
def test_chain_is_causal(fa, fp8):
    """A chain's masks are the causal one: bit by bit, where both take the same work (up to 16 rows)."""
    c = Cache([200, 33, 8], 2, 128, 16, fp8, seed=5)
    new, Hq = [8, 8, 8], 4
    o, lse = attend(fa, c, new, Hq, kind="chain")
    q = randn((24, Hq, 128), 3).cuda()
    o2, lse2 = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu_of(new), max_q=8, **c.scales)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("n", [4, 50])
def test_hidden_tokens_do_not_matter(fa, n):
    """Keys that no row sees may hold anything."""
    c = Cache([100 + n], 1, 128, 16, False, seed=1)
    bits = masks([n], 7)[0]
    bits[:, n - 1] = False                        # the last token is seen by none, itself among them
    tree = words_of([bits], n)
    q = randn((n, 4, 128), 2).cuda()
    args = dict(cu_seqlens=cu_of([n]), max_q=n, tree=tree)
    a = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, **args)
    page, slot = P.slot_of(c.table, 16, 0, 100 + n - 1)
    for x in (float("nan"), float("inf"), -float("inf")):
        c.k_pages[page, :, slot] = x
        b = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, **args)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert fa.get_device_error() == 0


@pytest.mark.parametrize("n,Hq", [(5, 2), (48, 8)])
def test_graph_and_stream(fa, n, Hq):
    """Masks and attention captured into a graph on another stream, replayed for another tree."""
    c = Cache([150 + n, n], 2, 128, 16, False, seed=6)
    q = randn((2, n, Hq, 128), 2).cuda()
    parents = torch.from_numpy(np.stack([parents_of(n, 1), parents_of(n, 2)])).cuda()
    args = (c.k_pages, c.v_pages, c.block_table, c.seq_lens)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        fa.fwd_paged(q, *args, tree=fa.tree_mask(parents)[0])          # (the first call of a kernel sets its limits)
    stream.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        mask, depth = fa.tree_mask(parents)
        o, lse = fa.fwd_paged(q, *args, tree=mask)
    for seed in (3, 4):
        parents.copy_(torch.from_numpy(np.stack([parents_of(n, seed), parents_of(n, seed + 9)])))
        graph.replay()
        torch.cuda.synchronize()
        want_mask, want_depth = fa.tree_mask(parents, stream=stream)
        want = fa.fwd_paged(q, *args, tree=want_mask, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(mask, want_mask) and torch.equal(depth, want_depth)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert fa.get_device_error() == 0


def test_binding_refusals(fa):
    c = Cache([40], 1, 64, 16, False)
    q = randn((1, 33, 1, 64), 1).cuda()
    args = (q, c.k_pages, c.v_pages, c.block_table, c.seq_lens)
    good = torch.zeros(1, 33, 2, dtype=torch.int32, device="cuda")
    for bad in (good[..., :1].contiguous(), good.float(), good.cpu(), good[0], good.expand(1, 33, 2).transpose(1, 2)):
        with pytest.raises(ValueError):
            fa.fwd_paged(*args, tree=bad)
    with pytest.raises(ValueError):
        fa.fwd_paged(*args, tree=good, causal=False)
    with pytest.raises(fa.FAError):
        fa.tree_mask(torch.zeros(1, 1025, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        fa.tree_mask(torch.zeros(4, dtype=torch.int32, device="cuda"), cu_of([4]), max_q=5)
    with pytest.raises(ValueError):
        fa.tree_mask(torch.zeros(4, dtype=torch.int64, device="cuda"), cu_of([4]))
    assert fa.get_device_error() == 0
