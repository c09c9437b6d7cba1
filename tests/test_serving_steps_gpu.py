"""The operators of speculative decoding and of eviction in a row, as a serving
program calls them, against a plain cache that is a list of rows."""

import numpy as np
import pytest
import torch

from oracle import paged as P

from paged_case import Cache, cu_of, randn
from parity import f64
from tree_case import check_rows, parents_of
from weights_case import lse_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


class Plain:
    """What the pages stand for: keys and values of each sequence [L, Hkv, D] in fp64."""

    def __init__(self, cache):
        self.lens = cache.lens
        self.kv = {x: [cache.rows(x, b).copy() for b in range(len(cache.lens))] for x in "kv"}

    def rows(self, name, b):
        return self.kv[name][b]

    def append(self, name, b, rows):
        self.kv[name][b] = np.concatenate([self.kv[name][b], rows])


def ints(x):
    return torch.tensor(np.array(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,Hq", [(6, 4), (40, 8)])
def test_speculative_step(fa, n, Hq, fp8):
    """Write a tree of drafts, attend with its masks, keep the accepted path, decode one
    token: the same as if only the accepted tokens had ever been there."""
    D, Hkv, page = 128, 2, 16
    past = [100, 17, 64, 0]
    c = Cache(past, Hkv, D, page, fp8, seed=3, cols=16, spare=60)
    # room for the drafts: more pages of each sequence
    free = iter(sorted(set(range(c.num_pages)) - set(c.table[c.table >= 0].tolist())))
    for b, L in enumerate(past):
        for j in range(-(-L // page), -(-(L + n + 1) // page)):
            c.table[b, j] = next(free)
    c.upload()
    plain = Plain(c)
    B = len(past)
    parents = [parents_of(n, 5 + b, far=3) for b in range(B)]
    mask, depth = fa.tree_mask(ints(parents))
    positions = ints(past).unsqueeze(1) + depth
    k, v, q = randn((B, n, Hkv, D), 1).cuda(), randn((B, n, Hkv, D), 2).cuda(), randn((B, n, Hq, D), 4).cuda()
    q, k = fa.rope(q, k, positions.contiguous())
    lens = ints([L + n for L in past])
    fa.cache_write(k, v, c.k_pages, c.v_pages, c.block_table, lens, **c.scales)
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, lens, tree=mask, **c.scales)
    assert fa.get_device_error() == 0

    def stored(x):
        return P.dequantise(*P.quantise(f64(x))) if fp8 else f64(x)

    sees = []
    for b in range(B):
        plain.append("k", b, stored(k[b]))
        plain.append("v", b, stored(v[b]))
        sees.append(P.tree_sees(P.tree_ancestors(parents[b])[0], past[b] + n))
    check_rows(o.view(B * n, Hq, D), lse.transpose(0, 1).reshape(Hq, -1), q.view(B * n, Hq, D), plain, [n] * B, sees,
               D ** -0.5)

    # the accepted path: the ancestors of some token, by number
    paths = [np.flatnonzero(P.tree_ancestors(parents[b])[0][n - 1 - b]) for b in range(B)]
    counts = [len(p) for p in paths]
    index = np.full((B, 1, max(counts)), -1, dtype=np.int32)
    for b, p in enumerate(paths):
        index[b, 0, :len(p)] = past[b] + p
        for x in "kv":
            plain.kv[x][b] = np.concatenate([plain.kv[x][b][:past[b]], plain.kv[x][b][past[b] + p]])
    fa.cache_keep(c.k_pages, c.v_pages, c.block_table, ints(index), ints(counts), ints(past), **c.scales)
    lens = [past[b] + counts[b] + 1 for b in range(B)]
    k, v, q = randn((B, 1, Hkv, D), 6).cuda(), randn((B, 1, Hkv, D), 7).cuda(), randn((B, 1, Hq, D), 8).cuda()
    fa.cache_write(k, v, c.k_pages, c.v_pages, c.block_table, ints(lens), **c.scales)
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, ints(lens), **c.scales)
    assert fa.get_device_error() == 0
    for b in range(B):
        plain.append("k", b, stored(k[b]))
        plain.append("v", b, stored(v[b]))
    check_rows(o.view(B, Hq, D), lse.transpose(0, 1).reshape(Hq, -1), q.view(B, Hq, D), plain, [1] * B,
               [np.ones((1, L), dtype=bool) for L in lens], D ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 30])
def test_eviction(fa, n, fp8):
    """Attend, add the weights up, choose, move together, attend from the next token:
    over what each head kept, and its sums went along."""
    D, Hkv, Hq, page, keep = 64, 2, 8, 32, 96
    lens = [400, 96, 131, 60]
    c = Cache(lens, Hkv, D, page, fp8, seed=5)
    plain = Plain(c)
    B = len(lens)
    q = randn((B * n, Hq, D), 1)
    args = dict(cu_seqlens=cu_of([n] * B), max_q=n)
    sums = torch.full(c.k_pages.shape[:3], float("nan"), device="cuda")
    _, lse = fa.fwd_paged(q.cuda(), c.k_pages, c.v_pages, c.block_table, c.seq_lens, **args, **c.scales)
    fa.cache_weights(q.cuda(), lse, c.k_pages, sums, c.block_table, c.seq_lens, decay=0.0, k_scale=c.k_scale, **args)
    before = sums.cpu().numpy()
    index, kept = fa.cache_select(sums, c.block_table, c.seq_lens, keep, first=2, recent=20)
    fa.cache_keep(c.k_pages, c.v_pages, c.block_table, index, kept, sums=sums, **c.scales)
    assert fa.get_device_error() == 0
    assert kept.tolist() == [min(L, keep) for L in lens]
    after = sums.cpu().numpy()
    ref = lse_of(q, c, [n] * B, True, D ** -0.5).numpy().astype(np.float64)
    for b, L in enumerate(lens):
        t = np.arange(L)
        w, _ = P.weights(f64(q[b * n:(b + 1) * n]), ref[:, b * n:(b + 1) * n], plain.rows("k", b), P.causal_sees(n, L, True),
                         D ** -0.5)
        got = before[c.table[b, t // page], :, t % page].T
        np.testing.assert_allclose(got, w, rtol=1e-4, atol=1e-7)      # (test_weights_gpu.py has the bounds)
        m = min(L, keep)
        for h in range(Hkv):
            at = index[b, h, :m].cpu().numpy()
            np.testing.assert_array_equal(at, P.select(got[h], keep, 2, 20))
            np.testing.assert_array_equal(after[c.table[b, t[:m] // page], h, t[:m] % page], got[h, at])
            for x in "kv":
                plain.kv[x][b][:m, h] = plain.kv[x][b][at, h]
        for x in "kv":
            plain.kv[x][b] = plain.kv[x][b][:m]
    # the next token, whose slot is behind the kept ones
    lens = [min(L, keep) + 1 for L in lens]
    cols = c.table.shape[1]
    for b, L in enumerate(lens):
        if c.table[b, (L - 1) // page] < 0 or (L - 1) // page >= cols:
            lens[b] = L - 1
    k, v, q = randn((B, Hkv, D), 6).cuda(), randn((B, Hkv, D), 7).cuda(), randn((B, Hq, D), 8).cuda()
    new = [int(L > min(x, keep)) for L, x in zip(lens, c.lens)]
    rows = np.flatnonzero(new)
    fa.cache_write(k[rows].contiguous(), v[rows].contiguous(), c.k_pages, c.v_pages, c.block_table, ints(lens),
                   cu_seqlens=cu_of(new), **c.scales)
    o, lse = fa.fwd_paged(q[rows].contiguous(), c.k_pages, c.v_pages, c.block_table, ints(lens), cu_seqlens=cu_of(new),
                          max_q=1, **c.scales)
    assert fa.get_device_error() == 0 and len(rows) >= 3
    for b in rows:
        for x, y in (("k", k), ("v", v)):
            one = f64(y[b:b + 1])
            plain.append(x, b, P.dequantise(*P.quantise(one)) if fp8 else one)
    check_rows(o, lse, q[rows], plain, new, [np.ones((m, L), dtype=bool) for m, L in zip(new, lens)], D ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_far_from_the_first(fa, fp8):
    """Pages whose elements lie behind the 2^31st: bit by bit what the same pages give at
    the front."""
    D, Hkv, Hq, page, far = 128, 8, 16, 64, 33000 * (2 if fp8 else 1)
    lens, B = [300, 129, 700], 3
    c = Cache(lens, Hkv, D, page, fp8, seed=6)
    assert far * Hkv * page * D > 2 ** 31
    big = {}
    for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
        x = getattr(c, name)
        if x is None:
            big[name] = None
            continue
        big[name] = torch.empty((far + c.num_pages, *x.shape[1:]), dtype=x.dtype, device="cuda")
        big[name].view(torch.uint8)[far:] = x.view(torch.uint8)
    table = torch.where(c.block_table >= 0, c.block_table + far, c.block_table)
    sums = torch.rand(c.k_pages.shape[:3], generator=torch.Generator().manual_seed(2)).cuda()
    far_sums = torch.empty((far + c.num_pages, Hkv, page), device="cuda")
    far_sums[far:] = sums

    def steps(k, v, ks, vs, table, sums):
        out = []
        for n in (2, 40):
            q = randn((B, n, Hq, D), n).cuda()
            mask, _ = fa.tree_mask(ints([parents_of(n, b) for b in range(B)]))
            out += fa.fwd_paged(q, k, v, table, c.seq_lens, tree=mask, k_scale=ks, v_scale=vs)
            _, lse = fa.fwd_paged(q, k, v, table, c.seq_lens, k_scale=ks, v_scale=vs)
            fa.cache_weights(q, lse, k, sums, table, c.seq_lens, k_scale=ks)
        out += fa.cache_select(sums, table, c.seq_lens, 100, first=1, recent=9)
        fa.cache_keep(k, v, table, out[-2], out[-1], k_scale=ks, v_scale=vs, sums=sums)
        assert fa.get_device_error() == 0
        return out

    near = steps(c.k_pages, c.v_pages, c.k_scale, c.v_scale, c.block_table, sums)
    there = steps(big["k_pages"], big["v_pages"], big["k_scale"], big["v_scale"], table, far_sums)
    for a, b in zip(near, there):
        assert torch.equal(a, b)
    for name, x in list(big.items()) + [("sums", far_sums)]:
        if x is not None:
            small = sums if name == "sums" else getattr(c, name)
            assert torch.equal(x[far:].contiguous().view(torch.uint8), small.view(torch.uint8)), name


def test_streams_side_by_side(fa):
    """Calls on two streams at once, each over its own cache, bit by bit as one after the other."""
    def case(seed):
        c = Cache([900, 333], 2, 64, 32, bool(seed % 2), seed=seed)
        q = randn((2, 40, 8, 64), seed).cuda()
        mask, _ = fa.tree_mask(ints([parents_of(40, seed), parents_of(40, seed + 9)]))
        return c, q, mask, torch.zeros(c.k_pages.shape[:3], device="cuda")

    def run(c, q, mask, sums):
        out = list(fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, tree=mask, **c.scales))
        _, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, **c.scales)
        fa.cache_weights(q, lse, c.k_pages, sums, c.block_table, c.seq_lens, k_scale=c.k_scale)
        fa.cache_weights(q[:, :1].contiguous(), lse[:, :, :1].contiguous(), c.k_pages, sums, c.block_table, c.seq_lens,
                         k_scale=c.k_scale)
        index, kept = fa.cache_select(sums, c.block_table, c.seq_lens, 64)
        fa.cache_keep(c.k_pages, c.v_pages, c.block_table, index, kept, sums=sums, **c.scales)
        return out + [index, kept, sums, c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8)]

    want = [[x.clone() for x in run(*case(s))] for s in (1, 2)]
    cases = [case(s) for s in (1, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for s, k in zip(streams, cases):
        with torch.cuda.stream(s):
            got.append(run(*k))
    torch.cuda.synchronize()
    assert fa.get_device_error() == 0
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
