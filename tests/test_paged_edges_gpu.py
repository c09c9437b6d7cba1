"""Attention over a paged cache where calls are unusual: pages that are missing,
values that are not finite, scales far apart, head groups that do not fill a
tile, shared pages, graphs, streams, short workspaces."""

import numpy as np
import pytest
import torch

from oracle import paged as P

from paged_case import Cache, check_attention, cu_of, randn
from parity import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


def run(fa, c, q, new, causal=True, table=None, **kw):
    """Packed call; (o, lse)."""
    kw.setdefault("max_q", max(new))
    return fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table if table is None else table, c.seq_lens, causal=causal,
                        cu_seqlens=cu_of(new), **c.scales, **kw)


def attend(fa, c, new, Hq, causal=True, seed=3, **kw):
    q = randn((sum(new), Hq, c.D), seed).cuda()
    o, lse = run(fa, c, q, new, causal, **kw)
    assert fa.get_device_error() == 0
    check_attention(o, lse, q, c, new, causal, kw.get("scale", c.D ** -0.5))
    return q, o, lse


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (10, 2), (7, 1), (48, 3), (100, 1), (128, 1)])
def test_chunks_of_head_groups(fa, Hq, Hkv, fp8):
    """Groups that leave rows of a tile without a token, up to one token a tile."""
    c = Cache([300, 40, 131], Hkv, 128, 32, fp8, seed=Hq)
    attend(fa, c, [45, 1, 66], Hq)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 128, 256, 512, 1024])
def test_page_sizes(fa, D, page, fp8):
    c = Cache([1, 700, 129, 256], 2, D, page, fp8, seed=page)
    attend(fa, c, [1, 50, 129, 2], 4)
    attend(fa, c, [1, 2, 1, 2], 4)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,n", [(1, 1), (1, 8), (4, 4), (8, 3), (5, 6), (8, 4), (16, 2)])
def test_few_rows(fa, group, n, D, fp8, causal):
    """1 to 32 rows of a sequence and head, on either side of the choice of kernel."""
    c = Cache([500, 1, 33, n, 0], 2, D, 64, fp8, seed=group + n)
    attend(fa, c, [n, 1, n, n, 1], 2 * group, causal)


@pytest.mark.parametrize("fp8", [False, True])
def test_dense_chunks_with_padded_entries(fa, fp8):
    """A dense batch whose entries are longer than, as long as and shorter than
    the new tokens, or empty."""
    n, lens = 40, [200, 40, 13, 0]
    c = Cache(lens, 2, 64, 16, fp8, seed=3)
    q = randn((4, n, 6, 64), 1).cuda()
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, **c.scales)
    assert fa.get_device_error() == 0
    check_attention(o.view(4 * n, 6, 64), lse.transpose(0, 1).reshape(6, -1), q.view(4 * n, 6, 64), c, [n] * 4, True,
                    64 ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
def test_chunks_of_many_sequences(fa, fp8):
    """1024 sequences, the most, some without new tokens and some without keys."""
    r = np.random.default_rng(2)
    new = r.integers(0, 60, 1024).tolist()
    lens = [int(m) if b % 7 == 0 else n + int(m) for b, (n, m) in enumerate(zip(new, r.integers(0, 90, 1024)))]
    c = Cache(lens, 1, 64, 16, fp8, seed=5)
    attend(fa, c, new, 1)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 20])
def test_long_sequence_in_small_pages(fa, new, fp8):
    c = Cache([50001], 1, 128, 16, fp8, seed=2)
    attend(fa, c, [new], 8)


def far_apart(c, seed, k_exp, v_exp):
    """Gives the cache rows whose scales differ by powers of two in [-exp, exp]."""
    for name, most in (("k", k_exp), ("v", v_exp)):
        e = torch.randint(-most, most + 1, c.scale_host[name].shape, generator=torch.Generator().manual_seed(seed))
        for b, n in enumerate(c.lens):
            first = sum(c.lens[:b])
            for t in range(n):
                p, s = P.slot_of(c.table, c.page, b, t)
                c.scale_host[name][p, :, s] = (c.scale_host[name][p, :, s].int() + e[p, :, s]).to(torch.uint8)
                c.value[name][first + t] *= 2.0 ** e[p, :, s].numpy().astype(np.float64)[:, None]
    c.upload()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 90])
def test_scales_far_apart(fa, D, new):
    """E4M3 rows whose scales differ by up to 2^20 (keys, 2^-20 of whose largest
    score is far below what LSE is held to) and 2^14 (values, exact)."""
    c = Cache([700, 300], 2, D, 32, True, seed=D)
    far_apart(c, 4, 7, 4)          # with the cache's own 2^-3 .. 2^3
    attend(fa, c, [new, new], 4, scale=2.0 ** -10)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 40])
def test_tiny_scale_and_queries_of_zero(fa, new, fp8):
    """The least scale, and rows of zeros: every key counts alike."""
    c = Cache([200], 1, 128, 16, fp8, seed=1)
    q = randn((new, 4, 128), 1).cuda()
    q[:, 1] = 0
    scale = 1e-37
    o, lse = run(fa, c, q, [new], scale=scale)
    assert fa.get_device_error() == 0
    check_attention(o, lse, q, c, [new], True, scale)
    with pytest.raises(fa.FAError):
        run(fa, c, q, [new], scale=1e-39)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 60])
def test_missing_pages_read_as_zeros(fa, D, new):
    """E4M3: a page number out of range counts as keys and values of zero, whatever
    the scales of the pages that are there."""
    c = Cache([200, 90], 1, D, 16, True, seed=7)
    free = sorted(set(range(c.num_pages)) - set(c.table[c.table >= 0].tolist()))
    # page 0 becomes one that no sequence has
    if 0 not in free:
        b, j = np.argwhere(c.table == 0)[0]
        c.table[b, j] = free[0]
        for t in list(c.host.values()) + list(c.scale_host.values()):
            t[free[0]] = t[0].clone()
    for byte in (255, 254):
        for t in c.scale_host.values():
            t[0] = byte
        c.upload()
        t = c.block_table.clone()
        t[0, 3], t[0, 12], t[1, 0] = -1, c.num_pages, 2 ** 31 - 1
        value = {n: v.copy() for n, v in c.value.items()}
        for v in c.value.values():
            v[48:64], v[192:200], v[200:216] = 0, 0, 0
        q = randn((2 * new, 4, D), 1).cuda()
        o, lse = run(fa, c, q, [new, new], table=t)
        assert fa.get_device_error() == 1
        check_attention(o, lse, q, c, [new, new], True, D ** -0.5)
        c.value = value


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_not_finite_values_show_where_they_are_seen(fa, new, fp8, what):
    """A NaN among a sequence's own values reaches the rows that see it and no
    other sequence; one in a query reaches that row alone."""
    c = Cache([300, 150], 2, 64, 32, fp8, seed=11)
    q = randn((2 * new, 8, 64), 2).cuda()
    if what == "q":
        q[new - 1, 5, 7] = float("nan")
    else:
        p, s = P.slot_of(c.table, c.page, 0, 120)
        if fp8:
            c.host[what][p, 1, s] = 0
            c.scale_host[what][p, 1, s] = 255
        else:
            c.host[what][p, 1, s] = float("nan")
        c.upload()
    o, lse = run(fa, c, q, [new, new])
    assert fa.get_device_error() == 0
    if what == "q":
        assert torch.isnan(o[new - 1, 5]).all() and torch.isnan(lse[5, new - 1])
        o[new - 1, 5] = 0
        assert torch.isfinite(o.float()).all()
    else:
        assert torch.isnan(o[:new, 4:]).all()                        # heads of the second key/value head
        assert torch.isfinite(o[:new, :4].float()).all()
        if what == "k":
            assert torch.isnan(lse[4:, :new]).all()
    c.lens = c.lens[1:]
    c.value = {n: v[300:] for n, v in c.value.items()}
    check_attention(o[new:], lse[:, new:], q[new:], c, [new], True, 64 ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 1, 1], [70, 1, 30]])
def test_shared_pages(fa, new, fp8):
    """Sequences with a common beginning, and a page that a sequence has twice."""
    c = Cache([160, 96, 64], 2, 128, 32, fp8, seed=4)
    c.table[1, :2] = c.table[0, :2]
    c.table[2, 1] = c.table[2, 0]
    c.block_table = torch.from_numpy(c.table).cuda()
    for v in c.value.values():
        v[160:224] = v[:64]
        v[160 + 96 + 32:] = v[160 + 96:160 + 96 + 32]
    attend(fa, c, new, 4)


@pytest.mark.parametrize("fp8", [False, True])
def test_results_repeat_whatever_the_workspace_holds(fa, fp8):
    new = [200, 1, 1, 40, 7, 1]
    c = Cache([5000, 3000, 17, 40, 900, 2500], 2, 128, 64, fp8, seed=6)
    q, o, lse = attend(fa, c, new, 8)
    need = fa.fwd_paged_workspace_size(6, 8, 2, sum(new), 128, packed=True, max_q=200)
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        o2, lse2 = run(fa, c, q, new, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new", [[1, 1], [100, 30]])
def test_workspace_and_counts_are_checked(fa, new):
    c = Cache([200, 100], 2, 128, 16, False)
    q = randn((sum(new), 8, 128), 1).cuda()
    need = fa.fwd_paged_workspace_size(2, 8, 2, sum(new), 128, packed=True, max_q=max(new))
    with pytest.raises(fa.FAError):
        run(fa, c, q, new, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        run(fa, c, q, new, workspace=torch.empty(need, dtype=torch.uint8))
    out = torch.full_like(q, 3.0)
    cu = cu_of([max(new) + 1, 0])                # more than max_q in one sequence
    wide = torch.cat([q, q])
    out = torch.full_like(wide, 3.0)
    fa.fwd_paged(wide, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu, max_q=max(new), out=out)
    assert fa.get_device_error() == 1 and (out == 3).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_two_graphs_and_two_streams_at_once(fa, fp8):
    """A decoding step and a chunk, each captured with a workspace of its own,
    replayed on two streams while eager calls of both run: the same bits."""
    cs = [Cache([3000, 700], 2, 128, 16, fp8, seed=1), Cache([2000, 300], 2, 128, 16, fp8, seed=2)]
    news = [[1, 1], [200, 60]]
    qs = [randn((sum(n), 8, 128), 5).cuda() for n in news]
    cus = [cu_of(n) for n in news]
    want = [run(fa, c, q, n) for c, q, n in zip(cs, qs, news)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    graphs, outs = [], []

    def call(i, **kw):
        c = cs[i]
        return fa.fwd_paged(qs[i], c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cus[i],
                            max_q=max(news[i]), **c.scales, **kw)

    for i in range(2):
        need = fa.fwd_paged_workspace_size(2, 8, 2, sum(news[i]), 128, packed=True, max_q=max(news[i]))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(i, workspace=ws))
        graphs.append((g, ws))
    for rep in range(5):
        for o, lse in outs:
            o.zero_()
            lse.zero_()
        torch.cuda.synchronize()
        eager = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i][0].replay()
            eager.append(call(1 - i, stream=s))
        torch.cuda.synchronize()
        for i in range(2):
            for got in (outs[i], eager[1 - i]):
                assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])
    assert fa.get_device_error() == 0


@pytest.mark.parametrize("interleaved,sections", [(False, [64]), (True, [30]), (False, [13, 20])])
def test_rope_write_attend_on_another_stream_in_place(fa, interleaved, sections):
    """The step of a serving loop on a stream that is not the current one, rope
    in place."""
    s = torch.cuda.Stream()
    new, lens = [60, 5], [60, 25]
    c = Cache(lens, 2, 128, 16, True, seed=8)
    T = sum(new)
    q, k, v = (randn((T, h, 128), 20 + h).cuda() for h in (8, 2, 2))
    pos = torch.tensor(np.stack([np.concatenate([np.arange(m - n, m) for n, m in zip(new, lens)])] * len(sections)),
                       dtype=torch.int32, device="cuda")
    want = [P.rope(f64(x), pos.cpu().numpy(), sections, 1e4, interleaved=interleaved) for x in (q, k)]
    s.wait_stream(torch.cuda.current_stream())
    fa.rope(q, k, pos, sections=sections, interleaved=interleaved, q_out=q, k_out=k, stream=s)
    fa.cache_write(k, v, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu_of(new), stream=s, **c.scales)
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu_of(new), stream=s,
                          **c.scales)
    s.synchronize()
    assert fa.get_device_error(s) == 0
    for x, w in zip((q, k), want):
        np.testing.assert_allclose(f64(x), w, rtol=2.0 ** -8, atol=1e-5)
    first = 0
    for b, n in enumerate(new):
        end = sum(lens[:b + 1])
        for name, x in (("k", k), ("v", v)):
            c.value[name][end - n:end] = P.dequantise(*P.quantise(f64(x[first:first + n])))
        first += n
    check_attention(o, lse, q, c, new, True, 128 ** -0.5)


def test_numbers_that_no_int_holds_are_refused(fa):
    c = Cache([20], 1, 64, 16, False)
    q = randn((4, 2, 64), 1).cuda()
    for max_q in (0, -1, 5, 2 ** 32 + 1):
        with pytest.raises(ValueError):
            run(fa, c, q, [4], max_q=max_q)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    for sections in ([0], [33], [2 ** 32 + 16]):
        with pytest.raises(ValueError):
            fa.rope(q, None, pos, sections=sections)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 1, 1], [90, 1, 200]])
def test_calls_behind_one_another(fa, new, fp8):
    """Copies, writes, attention calls and what reads their outputs, queued
    without a pause (a call may start while the one before still runs) and as a
    graph that begins with a copy: the bits of calls that wait for each other."""
    c = Cache([700, 64, 1500], 2, 128, 16, fp8, seed=9)
    T, cu = sum(new), cu_of(new)
    src = [[randn((T, h, 128), 10 * i + h).cuda() for h in (8, 2, 2)] for i in range(6)]
    q, k, v = (torch.empty_like(x) for x in src[0])

    def attention(x):
        return fa.fwd_paged(x, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu, max_q=max(new),
                            **c.scales)

    def step(pause):
        fa.cache_write(k, v, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu, **c.scales)
        pause()
        o, lse = attention(q)
        pause()
        o2, lse2 = attention(o)                # the outputs as the next call's queries
        pause()
        return o, lse, o2, lse2

    def series(pause):
        out = []
        for x in src:
            for to, y in zip((q, k, v), x):
                to.copy_(y)
            pause()
            out.append([t.clone() for t in step(pause)])
        torch.cuda.synchronize()
        return out

    want = series(torch.cuda.synchronize)
    for _ in range(5):
        for got, w in zip(series(lambda: None), want):
            assert all(torch.equal(a, b) for a, b in zip(got, w))
    source = [torch.empty_like(x) for x in src[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for to, y in zip((k, v, q), (source[1], source[2], source[0])):
            to.copy_(y)
        got = attention(q)                     # right behind a copy
        got2 = step(lambda: None)
    for x, w in zip(src, want):
        for to, y in zip(source, x):
            to.copy_(y)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got2, w))
    assert fa.get_device_error() == 0
    assert torch.isfinite(got[0].float()).all()
