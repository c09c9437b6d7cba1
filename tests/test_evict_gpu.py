"""Which tokens a head keeps, and the move of the kept rows, against plain forms."""

import numpy as np
import pytest
import torch

from oracle import paged as P

from paged_case import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


class Sums:
    """Sums of `lens` tokens in shuffled pages; every other slot holds a NaN."""

    def __init__(self, lens, Hkv, page, seed=0, make=None, cols=None):
        r = np.random.default_rng(seed)
        counts = [-(-n // page) for n in lens]
        self.lens, self.page = list(lens), page
        pages = sum(counts) + 2
        order = r.permutation(pages)
        self.table = np.full((len(lens), max(1, max(counts)) if cols is None else cols), -1, dtype=np.int32)
        self.host = np.full((pages, Hkv, page), np.nan, dtype=np.float32)
        self.rows, at = [], 0
        make = make or (lambda r, shape: r.random(shape) ** 6)
        for b, n in enumerate(lens):
            self.table[b, :counts[b]] = order[at:at + counts[b]]
            at += counts[b]
            x = make(r, (Hkv, n)).astype(np.float32)
            t = np.arange(n)
            self.host[self.table[b, t // page], :, t % page] = x.T
            self.rows.append(x)
        self.sums = torch.from_numpy(self.host).cuda()
        self.block_table = torch.from_numpy(self.table).cuda()
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def check(self, fa, keep, first=0, recent=0, **kw):
        index, kept = fa.cache_select(self.sums, self.block_table, self.seq_lens, keep, first, recent, **kw)
        assert fa.get_device_error() == 0
        got, counts = index.cpu().numpy(), kept.cpu().numpy()
        for b, rows in enumerate(self.rows):
            assert counts[b] == min(self.lens[b], keep)
            for h, x in enumerate(rows):
                want = P.select(x, keep, first, recent)
                np.testing.assert_array_equal(got[b, h, :len(want)], want)
                assert (got[b, h, len(want):] == -1).all()
        return index, kept


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("keep,first,recent", [(1, 0, 0), (7, 0, 7), (40, 4, 10), (40, 20, 20), (333, 1, 0), (5000, 3, 100)])
def test_select(fa, keep, first, recent, page):
    Sums([0, 1, 39, 40, 41, 1000, 4097], 3, page, seed=keep).check(fa, keep, first, recent)


@pytest.mark.parametrize("make", [
    lambda r, s: np.round(r.random(s) * 3),                                         # mostly equal
    lambda r, s: np.zeros(s), lambda r, s: -np.zeros(s) * np.sign(r.random(s) - 0.5),
    lambda r, s: r.standard_normal(s) * 10.0 ** r.integers(-40, 38, s),               # subnormals, both signs
    lambda r, s: np.where(r.random(s) < 0.3, np.nan, np.where(r.random(s) < 0.5, np.inf, -np.inf)),
    lambda r, s: 1 + np.round(r.random(s) * 4) * 2.0 ** -23])                        # apart in the last bits alone
def test_select_values(fa, make):
    s = Sums([700, 6000, 33], 2, 32, seed=5, make=make)
    for keep in (1, 32, 100, 600, 5999):
        s.check(fa, keep, min(2, keep // 2), keep // 3)


@pytest.mark.parametrize("L", [16384, 131073, 900001])
def test_select_long(fa, L):
    """More tokens than a cluster has room for are read again in each round."""
    s = Sums([L, 77], 1, 1024, seed=L)
    s.check(fa, L // 5, 16, 1000)
    s.check(fa, L - 1)


@pytest.mark.parametrize("L,B", [(900, 40), (3000, 14)])
def test_select_many(fa, L, B):
    """More heads than two blocks an SM, of short sequences and of longer ones."""
    Sums([L] * (B - 1) + [5], 32, 16, seed=1).check(fa, 100, 1, 30)


def test_select_bad_input(fa):
    s = Sums([100, 50], 2, 16, seed=3)
    lens = torch.tensor([s.table.shape[1] * 16 + 1, 50], dtype=torch.int32, device="cuda")
    for bad in (lens, torch.tensor([-1, 50], dtype=torch.int32, device="cuda")):
        index, kept = fa.cache_select(s.sums, s.block_table, bad, 20)
        assert fa.get_device_error() == 1
        assert kept.tolist() == [0, 20] and (index[0] == -1).all()
        for h in range(2):
            np.testing.assert_array_equal(index[1, h].cpu().numpy(), P.select(s.rows[1][h], 20, 0, 0))
    for page in (-3, s.host.shape[0], 2 ** 31 - 1):
        t = s.block_table.clone()
        t[0, 2] = page
        index, _ = fa.cache_select(s.sums, t, s.seq_lens, 20)
        assert fa.get_device_error() == 1
        for h in range(2):                          # its tokens' sums read as zero
            x = s.rows[0][h].copy()
            x[32:48] = 0
            np.testing.assert_array_equal(index[0, h].cpu().numpy(), P.select(x, 20, 0, 0))


def lists(lens, heads, keep, first, recent, seed):
    """Ascending random tokens, the first and the last among them: [B, heads, most], counts."""
    r = np.random.default_rng(seed)
    counts = [min(n, keep) for n in lens]
    index = np.full((len(lens), heads, max(1, max(counts))), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for h in range(heads):
            index[b, h, :counts[b]] = P.select(r.random(n).astype(np.float32), keep, first, recent)
    return index, counts


def raw(c, sums):
    out = c.raw()
    return [t.numpy().copy() for t in out] + ([] if sums is None else [sums.cpu().numpy().view(np.int32).copy()])


def check_keep(fa, c, index, counts, start=None, sums=True, stream=None):
    """cache_keep on cache c; every slot of every page is compared."""
    S = None
    if sums:
        g = torch.Generator().manual_seed(1)
        S = torch.rand(c.k_pages.shape[:3], generator=g).cuda()
    before = raw(c, S)
    dev = lambda x: torch.tensor(np.array(x), dtype=torch.int32, device="cuda")
    fa.cache_keep(c.k_pages, c.v_pages, c.block_table, dev(index), dev(counts), None if start is None else dev(start),
                  sums=S, **c.scales)
    assert fa.get_device_error() == 0
    after = raw(c, S)
    for x, y in zip(before, after):
        want = x.copy()
        for b, n in enumerate(counts):
            i = np.arange(n)
            to = i + (0 if start is None else start[b])
            for h in range(c.Hkv):
                of = index[b, 0 if index.shape[1] == 1 else h, :n]
                want[c.table[b, to // c.page], h, to % c.page] = x[c.table[b, of // c.page], h, of % c.page]
        np.testing.assert_array_equal(y, want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,keep,first,recent", [(16, 5, 1, 2), (16, 100, 0, 0), (64, 300, 4, 32), (1024, 700, 0, 700)])
def test_keep(fa, page, keep, first, recent, D, fp8):
    lens = [0, 1, 4, 90, 333, 1111]
    c = Cache(lens, 2, D, page, fp8, seed=keep)
    check_keep(fa, c, *lists(lens, 2, keep, first, recent, keep))
    check_keep(fa, c, *lists(lens, 1, keep, first, recent, keep + 1), sums=False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hkv,D", [(1, 128), (1, 64), (2, 128), (20, 64)])
def test_keep_long(fa, Hkv, D, fp8):
    """Many tiles, by clusters of several blocks; shifts by one row and by many."""
    L = 9000 if Hkv < 20 else 1500
    c = Cache([L], Hkv, D, 32, fp8, seed=D)
    index, counts = lists([L], Hkv, L - 1, 0, 0, 3)           # one evicted: every row behind it moves by one
    check_keep(fa, c, index, counts)
    check_keep(fa, c, *lists([L], Hkv, L // 2, 3, 100, 4))


@pytest.mark.parametrize("fp8", [False, True])
def test_keep_many(fa, fp8):
    """As many lists as leave each one block, and some tiles each."""
    lens = [600 - 2 * b for b in range(60)]
    c = Cache(lens, 4, 64, 16, fp8, seed=3)
    check_keep(fa, c, *lists(lens, 4, 550, 1, 7, 5))


@pytest.mark.parametrize("fp8", [False, True])
def test_keep_accepted(fa, fp8):
    """Accepted drafts of a step: some tokens behind `start`, none, all of them."""
    lens = [40, 17, 200, 64, 33]
    c = Cache(lens, 4, 128, 16, fp8, seed=2)
    start = [30, 16, 150, 60, 33]
    acc = [[30, 33, 38], [], [151, 152, 160, 161, 199], [60, 61, 62, 63], []]
    index = np.full((5, 1, 6), -1, dtype=np.int32)
    for b, a in enumerate(acc):
        index[b, 0, :len(a)] = a
    check_keep(fa, c, index, [len(a) for a in acc], start)


def test_keep_bad_input(fa):
    c = Cache([40, 60], 2, 64, 16, False, seed=1, junk=0.0)
    before = raw(c, None)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    good = [[1, 5, 9, 20], [0, 2, 3, 50]]
    cap = c.table.shape[1] * 16
    for bad in ([1, 5, 5, 20], [5, 1, 9, 20], [-1, 5, 9, 20], [1, 5, 9, cap], [1, 5, 9, 2 ** 31 - 1]):
        c.upload()
        index = dev([[good[0], bad], [good[1], good[1]]])         # nothing of the bad list moves, the others do
        fa.cache_keep(c.k_pages, c.v_pages, c.block_table, index, dev([4, 4]))
        assert fa.get_device_error() == 1
        after = raw(c, None)
        for x, y in zip(before, after):
            want = x.copy()
            for b, h, rows in ((0, 0, good[0]), (1, 0, good[1]), (1, 1, good[1])):
                for i, t in enumerate(rows):
                    want[c.table[b, i // 16], h, i % 16] = x[c.table[b, t // 16], h, t % 16]
            np.testing.assert_array_equal(y, want)
    index = dev([[good[0]], [good[1]]])
    for counts, start in (([5, -1], None), ([4, 4], [-1, 1]), ([4, 4], [2, 1])):
        c.upload()
        fa.cache_keep(c.k_pages, c.v_pages, c.block_table, index, dev(counts), None if start is None else dev(start))
        assert fa.get_device_error() == 1
        for x, y in zip(before, raw(c, None)):
            np.testing.assert_array_equal(x, y)
    c.upload()
    t = c.block_table.clone()
    t[0, 0] = c.num_pages
    fa.cache_keep(c.k_pages, c.v_pages, t, index, dev([4, 0]))     # a bad page: its tokens stay
    assert fa.get_device_error() == 1
    for x, y in zip(before, raw(c, None)):
        np.testing.assert_array_equal(x, y)


def test_graph_and_stream(fa):
    """Selection and move captured into a graph on another stream, replayed over other sums."""
    s = Sums([600, 350], 2, 16, seed=4)
    c = Cache([600, 350], 2, 64, 16, False, seed=4)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        fa.cache_select(s.sums, s.block_table, s.seq_lens, 100, 2, 20)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        index, kept = fa.cache_select(s.sums, s.block_table, s.seq_lens, 100, 2, 20)
        fa.cache_keep(c.k_pages, c.v_pages, s.block_table, index, kept, sums=s.sums)
    k, v = c.k_pages.clone(), c.v_pages.clone()
    for seed in (7, 8):
        c.k_pages.copy_(k)
        c.v_pages.copy_(v)
        x = torch.rand(s.sums.shape, generator=torch.Generator().manual_seed(seed)).cuda()
        s.sums.copy_(x)
        before = raw(c, x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert fa.get_device_error() == 0
        host = x.cpu().numpy()
        for y, z in zip(before, raw(c, s.sums)):
            want = y.copy()
            for b, n in enumerate([600, 350]):
                t = np.arange(n)
                for h in range(2):
                    of = P.select(host[s.table[b, t // 16], h, t % 16], 100, 2, 20)
                    np.testing.assert_array_equal(index[b, h].cpu().numpy(), of)
                    to = np.arange(100)
                    want[s.table[b, to // 16], h, to % 16] = y[s.table[b, of // 16], h, of % 16]
            np.testing.assert_array_equal(z, want)


def test_binding_refusals(fa):
    c = Cache([40], 2, 64, 16, True)
    sums = torch.zeros(c.k_pages.shape[:3], device="cuda")
    index, counts = torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    args = (c.k_pages, c.v_pages, c.block_table)
    for kw in (dict(sums=sums[:-1].contiguous()), dict(sums=sums.double()), dict(start=counts.long()),
               dict(start=torch.ones(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            fa.cache_keep(*args, index, counts, **c.scales, **kw)
    with pytest.raises(ValueError):
        fa.cache_keep(*args, index, counts)                       # E4M3 pages without scales
    with pytest.raises(ValueError):
        fa.cache_keep(*args, index.expand(2, 2, 4).contiguous(), counts, **c.scales)
    with pytest.raises(ValueError):
        fa.cache_keep(*args, index[:, :1].expand(1, 3, 4).contiguous(), counts, **c.scales)
    for kw in (dict(keep=0), dict(keep=4, first=5), dict(keep=4, first=2, recent=3), dict(keep=4, recent=-1)):
        with pytest.raises(ValueError):
            fa.cache_select(sums, c.block_table, c.seq_lens, **kw)
    with pytest.raises(ValueError):
        fa.cache_select(sums.half(), c.block_table, c.seq_lens, 4)
    assert fa.get_device_error() == 0


def test_long_selection_in_a_graph(fa):
    """A selection by clusters of 16 blocks, first called while a graph is captured."""
    s = Sums([150001], 1, 64, seed=6)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        index, kept = fa.cache_select(s.sums, s.block_table, s.seq_lens, 3000, 4, 500)
    for _ in range(2):
        index.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(index[0, 0].cpu().numpy(), P.select(s.rows[0][0], 3000, 4, 500))
    assert kept.tolist() == [3000] and fa.get_device_error() == 0
