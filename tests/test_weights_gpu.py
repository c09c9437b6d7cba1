"""Sums of the attention weights that a paged cache's keys get, against fp64."""

import numpy as np
import pytest
import torch

from paged_case import Cache, cu_of, randn
from weights_case import check, lse_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


LENS = [1, 15, 16, 17, 100, 128, 129, 333, 700]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_single_tokens(fa, D, page, fp8):
    c = Cache(LENS, 2, D, page, fp8, seed=page + D)
    check(fa, c, [1] * len(LENS), 8, dense=True)
    check(fa, c, [1] * len(LENS), 2, causal=False, decay=0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 128, 512])
@pytest.mark.parametrize("new,Hq", [([40, 300, 17, 129, 64], 4), ([150, 20, 1, 5, 130], 6)])
def test_chunks(fa, new, Hq, page, D, fp8):
    c = Cache([40, 333, 700, 129, 513], 2, D, page, fp8, seed=page + D)
    check(fa, c, new, Hq)
    check(fa, c, new, Hq, causal=False, decay=0.9)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (5, 5), (14, 2), (16, 1), (24, 1), (128, 1)])
@pytest.mark.parametrize("fp8", [False, True])
def test_head_groups(fa, Hq, Hkv, fp8):
    c = Cache([70, 3, 300], Hkv, 128, 32, fp8, seed=Hq)
    check(fa, c, [1, 1, 1], Hq, dense=True)
    check(fa, c, [50, 3, 2], Hq, max_q=53)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("most", [2, 90])
@pytest.mark.parametrize("causal", [False, True])
def test_ragged(fa, most, causal, fp8):
    """Sequences without new tokens, without keys, with fewer keys than tokens; rows
    behind the last sequence hold anything."""
    new = [min(n, most) for n in (1, 0, 40, 64, 2, 9, 90)]
    lens = [300, 55, 40, 65, 0, 1, 31]
    c = Cache(lens, 2, 128, 16, fp8, seed=4)
    q = randn((sum(new) + 5, 4, 128), 3)
    q[sum(new):] = float("nan")
    check(fa, c, new, 4, causal=causal, tail=5, q=q)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [2, 60])
def test_rows_without_weights(fa, n, fp8):
    """Rows whose LSE is -inf give nothing; decay 0 starts anew, whatever the old sums hold."""
    c = Cache([200], 2, 64, 16, fp8, seed=6)
    q = randn((n, 8, 64), 5)
    lse = lse_of(q, c, [n], True, 0.125)
    lse[::3, ::2] = -float("inf")
    check(fa, c, [n], 8, q=q, lse=lse, scale=0.125)
    sums = torch.full(c.k_pages.shape[:3], float("nan"), device="cuda")
    fa.cache_weights(q.cuda(), lse.cuda(), c.k_pages, sums, c.block_table, c.seq_lens, decay=0.0, cu_seqlens=cu_of([n]),
                     k_scale=c.k_scale)
    assert int(torch.isfinite(sums).sum()) == 2 * 200


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,Hq", [(1, 4), (500, 4), (40, 4)])
def test_long(fa, n, Hq, fp8):
    """Units and rows enough for every thread block to have several."""
    c = Cache([9001, 3000], 1, 128, 128, fp8, seed=8)
    check(fa, c, [n, n // 2 + 1], Hq)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("L", [90, 600])
def test_many_units(fa, L, fp8):
    """A dozen units or more for every thread block, of one tile of rows each and of two."""
    c = Cache([L] * (300 if L < 256 else 100), 8, 64, 64, fp8, seed=2)
    check(fa, c, [9 + b % 2 * 5 for b in range(len(c.lens))], 32)


@pytest.mark.parametrize("new", [1, 100])
def test_far_scores(fa, new):
    """Large scores, far from the LSE and near it, and a scale of its own."""
    for fp8 in (False, True):
        c = Cache([500], 1, 128, 32, fp8, seed=4)
        q = (randn((new, 4, 128), 6) * 8).to(torch.bfloat16)
        check(fa, c, [new], 4, q=q)
        check(fa, c, [new], 4, scale=0.01)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 70])
def test_sums_of_an_attention_call(fa, n, fp8):
    """With the LSE that fwd_paged gives, every row's weights add up to one; and the
    call repeats bit by bit."""
    c = Cache([900, 333], 2, 128, 64, fp8, seed=9)
    q = randn((2, n, 8, 128), 1).cuda()
    args = (c.block_table, c.seq_lens)
    _, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, *args, **c.scales)
    sums = torch.zeros(c.k_pages.shape[:3], device="cuda")
    again = torch.zeros_like(sums)
    for s in (sums, again):
        fa.cache_weights(q, lse, c.k_pages, s, *args, k_scale=c.k_scale)
    assert fa.get_device_error() == 0
    assert torch.equal(sums, again)
    # LSE and weights are off by 2^-20 or so each, see the tolerances of both
    np.testing.assert_allclose(sums.double().sum((0, 2)).cpu().numpy(), [2 * n * 4] * 2, rtol=1e-4)


@pytest.mark.parametrize("n,Hq", [(1, 4), (9, 3), (30, 4), (60, 3)])
def test_keys_that_are_not_finite(fa, n, Hq):
    """They reach their own sums alone: also where the group leaves columns of a tile
    without rows, and keys share a tile with them."""
    c = Cache([300], 1, 128, 16, False, seed=6)
    q, lse = randn((1, n, Hq, 128), 2).cuda(), torch.full((1, Hq, n), 5.0, device="cuda")
    want = torch.zeros(c.k_pages.shape[:3], device="cuda")
    fa.cache_weights(q, lse, c.k_pages, want, c.block_table, c.seq_lens)
    for x in (float("nan"), float("inf"), -float("inf")):
        c.upload()
        got = torch.zeros_like(want)
        for t in (7, 130):
            c.k_pages[c.table[0, t // 16], 0, t % 16, 5] = x
        fa.cache_weights(q, lse, c.k_pages, got, c.block_table, c.seq_lens)
        for t in (7, 130):
            got[c.table[0, t // 16], 0, t % 16] = want[c.table[0, t // 16], 0, t % 16]
        assert torch.equal(got, want)
    assert fa.get_device_error() == 0


def test_bad_input(fa):
    for n in (1, 40):
        c = Cache([40, 60], 1, 64, 16, False, seed=1, junk=0.0)
        q, lse = randn((2, n, 4, 64), 1).cuda(), torch.zeros(2, 4, n, device="cuda")
        sums = torch.full(c.k_pages.shape[:3], 3.0, device="cuda")
        for lens in ([41, -1], [65, 20]):
            fa.cache_weights(q, lse, c.k_pages, sums, c.block_table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
            assert fa.get_device_error() == 1 and (sums == 3).all()
        for cu in ([0, 2 * n, n], [1, n, 2 * n], [0, n, 2 * n + 1]):
            fa.cache_weights(q.view(2 * n, 4, 64), lse.view(4, 2 * n), c.k_pages, sums, c.block_table, c.seq_lens,
                             cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
            assert fa.get_device_error() == 1 and (sums == 3).all()
        for page in (-5, c.num_pages, 2 ** 31 - 1):
            t = c.block_table.clone()
            t[0, 1] = page
            got = sums.clone()
            fa.cache_weights(q, lse, c.k_pages, got, t, c.seq_lens)
            assert fa.get_device_error() == 1
            good = sums.clone()
            fa.cache_weights(q, lse, c.k_pages, good, c.block_table, c.seq_lens)
            assert fa.get_device_error() == 0
            good[c.table[0, 1]] = 3.0                      # the bad page's tokens get no sum, the others theirs
            assert torch.equal(got, good)


@pytest.mark.parametrize("n", [1, 50])
def test_graph_and_stream(fa, n):
    c = Cache([150 + n, 90 + n], 2, 128, 16, False, seed=6)
    q, lse = randn((2, n, 8, 128), 2).cuda(), torch.zeros(2, 8, n, device="cuda")
    sums = torch.zeros(c.k_pages.shape[:3], device="cuda")
    args = (c.block_table, c.seq_lens)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        fa.cache_weights(q, lse, c.k_pages, sums, *args)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        _, got = fa.fwd_paged(q, c.k_pages, c.v_pages, *args)
        fa.cache_weights(q, got, c.k_pages, sums, *args)
    want = torch.zeros_like(sums)
    sums.zero_()
    torch.cuda.synchronize()
    for seed in (3, 4):
        q.copy_(randn((2, n, 8, 128), seed))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, *args, stream=stream)
        fa.cache_weights(q, lse, c.k_pages, want, *args, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(sums, want)
    assert fa.get_device_error() == 0


def test_binding_refusals(fa):
    c = Cache([40], 2, 64, 16, True)
    q, lse = randn((1, 3, 4, 64), 1).cuda(), torch.zeros(1, 4, 3, device="cuda")
    sums = torch.zeros(c.k_pages.shape[:3], device="cuda")
    rest = (c.block_table, c.seq_lens)
    good = dict(k_scale=c.k_scale)
    for bad in (lse[0], lse.double(), lse.transpose(1, 2), lse.cpu()):
        with pytest.raises(ValueError):
            fa.cache_weights(q, bad, c.k_pages, sums, *rest, **good)
    for bad in (sums[1:].contiguous(), sums.half(), sums.cpu(), sums.transpose(0, 1)):
        with pytest.raises(ValueError):
            fa.cache_weights(q, lse, c.k_pages, bad, *rest, **good)
    with pytest.raises(ValueError):
        fa.cache_weights(q, lse, c.k_pages, sums, *rest)                 # E4M3 pages without scales
    for kw in (dict(decay=-1.0), dict(scale=0.0), dict(decay=float("nan"))):
        with pytest.raises(fa.FAError):
            fa.cache_weights(q, lse, c.k_pages, sums, *rest, **good, **kw)
    assert fa.get_device_error() == 0
