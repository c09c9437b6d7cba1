"""Attention of new tokens over a paged cache, the cache's writes and its
read-back, against plain fp64 forms."""

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


def clean(fa):
    assert fa.get_device_error() == 0


def attend(fa, c, new, Hq, causal, seed=3, dense=False, **kw):
    q = randn((sum(new), Hq, c.D), seed).cuda()
    scale = c.D ** -0.5
    args = (c.k_pages, c.v_pages, c.block_table, c.seq_lens)
    if dense:
        o, lse = fa.fwd_paged(q.view(len(new), new[0], Hq, c.D), *args, causal=causal, **c.scales, **kw)
        o, lse = o.view(q.shape), lse.transpose(0, 1).reshape(Hq, -1)
    else:
        o, lse = fa.fwd_paged(q, *args, causal=causal, cu_seqlens=cu_of(new), **c.scales, **kw)
    clean(fa)
    check_attention(o, lse, q, c, new, causal, scale)
    return o, lse


LENS = [1, 15, 16, 17, 100, 128, 129, 333]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_single_tokens(fa, D, page, fp8):
    c = Cache(LENS, 2, D, page, fp8, seed=page + D)
    attend(fa, c, [1] * len(LENS), 8, True, dense=True)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (5, 5), (14, 2), (16, 1), (24, 1), (128, 1)])
@pytest.mark.parametrize("fp8", [False, True])
def test_head_groups(fa, Hq, Hkv, fp8):
    c = Cache([70, 3, 200], Hkv, 128, 32, fp8, seed=Hq)
    attend(fa, c, [1, 1, 1], Hq, True, dense=True)
    attend(fa, c, [5, 3, 2], Hq, True, max_q=5)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_chunks(fa, D, fp8, causal):
    """From one token to more than a tile of rows; a chunk that is the whole
    sequence, and one with more new tokens than keys (rows that see nothing)."""
    new = [1, 40, 129, 0, 64, 17, 300, 9]
    lens = [300, 40, 400, 55, 65, 3, 513, 0]
    c = Cache(lens, 2, D, 64, fp8, seed=D)
    attend(fa, c, new, 4, causal)


@pytest.mark.parametrize("fp8", [False, True])
def test_no_keys_at_all(fa, fp8):
    c = Cache([0, 0], 1, 128, 16, fp8)
    o, lse = attend(fa, c, [1, 1], 4, True, dense=True)
    assert not o.any() and torch.isinf(lse).all()


@pytest.mark.parametrize("new", [1, 70])
def test_one_long_sequence_is_split(fa, new):
    """A single sequence's keys are split over all thread blocks and joined;
    the result does not depend on the workspace's contents, and repeats bit by
    bit."""
    c = Cache([9001], 1, 128, 128, False, seed=8)
    a = attend(fa, c, [new], 8, True)
    need = fa.fwd_paged_workspace_size(1, 8, 1, new, 128, packed=True)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    b = attend(fa, c, [new], 8, True, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 1, 1], [30, 1, 90]])
def test_rows_behind_the_last_sequence_stay(fa, new, fp8):
    c = Cache([100, 31, 90], 2, 64, 16, fp8)
    total = sum(new) + 9
    q = randn((total, 4, 64), 5).cuda()
    q[sum(new):] = float("nan")
    out, lse = torch.full_like(q, 7.0), torch.full((4, total), 7.0, device="cuda")
    fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu_of(new), max_q=max(new), out=out,
                 lse=lse, **c.scales)
    clean(fa)
    assert (out[sum(new):] == 7).all() and (lse[:, sum(new):] == 7).all()
    check_attention(out[:sum(new)], lse[:, :sum(new)], q[:sum(new)], c, new, True, 64 ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 200])
def test_large_scores_and_values_far_apart(fa, new, fp8):
    """Rows' maxima that move late and by much, and values of unlike size."""
    c = Cache([700], 1, 128, 32, fp8, seed=4)
    q = (randn((new, 4, 128), 6) * 8).cuda()
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu_of([new]), **c.scales)
    clean(fa)
    check_attention(o, lse, q, c, [new], True, 128 ** -0.5)


def test_bad_input_is_reported(fa):
    c = Cache([40, 20], 1, 128, 16, False, junk=0.0)
    q = randn((2, 1, 4, 128), 1).cuda()
    args = (q, c.k_pages, c.v_pages)
    out = torch.full_like(q, 3.0)
    for lens in ([41, -1], [49, 20]):          # negative; more than the table holds
        fa.fwd_paged(*args, c.block_table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out=out)
        assert fa.get_device_error() == 1
        assert (out == 3).all()
    packed = q.view(2, 4, 128)
    for cu in ([0, 2, 1], [1, 1, 2], [0, 1, 3], [0, 2, 2]):      # order, start, end, more than max_q
        fa.fwd_paged(packed, c.k_pages, c.v_pages, c.block_table, c.seq_lens,
                     cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q=1, out=out.view(2, 4, 128))
        assert fa.get_device_error() == 1
        assert (out == 3).all()
    for page in (-5, c.num_pages, 2 ** 31 - 1):
        t = c.block_table.clone()
        t[0, 1] = page
        o, _ = fa.fwd_paged(*args, t, c.seq_lens)
        assert fa.get_device_error() == 1
        assert torch.isfinite(o.float()).all()                   # the page reads as zeros
        k, v = fa.cache_read(c.k_pages, c.v_pages, t, cu_of(c.lens), 60)
        assert fa.get_device_error() == 1
        assert not k[16:32].any() and k[:16].any() and not v[16:32].any()
    clean(fa)


# ---------------------------------------------------------- write and read --

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,new,dense", [(16, [1, 1, 1, 1], True), (16, [40, 0, 1, 33], False),
                                            (128, [300, 5, 129, 1], False), (1024, [64] * 3, True)])
def test_write_then_read(fa, D, page, new, dense, fp8):
    lens = [n + p for n, p in zip(new, [7, 50, 0, 20])]
    Hkv = 3
    c = Cache(lens, Hkv, D, page, fp8, seed=1)
    before = c.raw()
    x = {"k": randn((sum(new), Hkv, D), 11, 30.0), "v": randn((sum(new), Hkv, D), 12, 1e-3)}
    dev = {n: t.cuda() for n, t in x.items()}
    if dense:
        dev = {n: t.view(len(new), new[0], Hkv, D) for n, t in dev.items()}
    fa.cache_write(dev["k"], dev["v"], c.k_pages, c.v_pages, c.block_table, c.seq_lens,
                   cu_seqlens=None if dense else cu_of(new), **c.scales)
    clean(fa)
    # exactly the new slots changed, to exactly the expected bits
    want = [t.clone() for t in before]
    for i, name in enumerate("kv"):
        codes, scale = P.quantise(f64(x[name])) if fp8 else (x[name].view(torch.int16).numpy(), None)
        first = 0
        for b, n in enumerate(new):
            for t in range(n):
                p, s = P.slot_of(c.table, page, b, lens[b] - n + t)
                want[i][p, :, s] = torch.from_numpy(codes[first + t])
                if fp8:
                    want[2 + i][p, :, s] = torch.from_numpy(scale[first + t])
            first += n
    for got, w in zip(c.raw(), want):
        assert torch.equal(got, w)
    # read back
    k, v = fa.cache_read(c.k_pages, c.v_pages, c.block_table, cu_of(lens), sum(lens) + 3, **c.scales)
    clean(fa)
    for name, got, i in (("k", k, 0), ("v", v, 1)):
        for b, n in enumerate(lens):
            first = sum(lens[:b])
            rows = P.gather(want[i].numpy(), c.table, b, n)
            if fp8:
                ref = P.dequantise(rows, P.gather(want[2 + i].numpy(), c.table, b, n))
            else:
                ref = f64(torch.from_numpy(rows).view(torch.bfloat16))
            np.testing.assert_array_equal(f64(got[first:first + n]), ref)


def test_quantised_values_at_every_scale(fa):
    """Rows from the smallest to the largest BF16 values, zeros, ties, and rows
    that are not finite; the codes and scales are the oracle's bit by bit, and
    every code reads back exactly."""
    D, n = 64, 300
    g = torch.Generator().manual_seed(3)
    x = torch.randn(n, 1, D, generator=g) * torch.exp2(torch.linspace(-140, 127, n)).view(n, 1, 1)
    x = x.clamp(-3.3e38, 3.3e38)
    x[5] = 0
    x[6, 0, 3], x[7, 0, 60], x[8, 0, 0] = float("nan"), float("inf"), -float("inf")
    x[9], x[10] = 3.3895313892515355e38, 448.0
    x[11, 0] = torch.from_numpy(P.e4m3_grid()[60:124]).float()                       # on the grid
    x[12, 0, :62] = torch.from_numpy((P.e4m3_grid()[60:122] + P.e4m3_grid()[61:123]) / 2).float()   # ties
    x[12, 0, 62:] = 448
    x = x.to(torch.bfloat16)
    c = Cache([n], 1, D, 16, True, seed=2)
    fa.cache_write(x.cuda(), x.flip(0).contiguous().cuda(), c.k_pages, c.v_pages, c.block_table, c.seq_lens,
                   cu_seqlens=cu_of([n]), **c.scales)
    clean(fa)
    raw = c.raw()
    codes, scale = P.quantise(f64(x))
    np.testing.assert_array_equal(P.gather(raw[2].numpy(), c.table, 0, n), scale)
    np.testing.assert_array_equal(P.gather(raw[0].numpy(), c.table, 0, n), codes)
    k, v = fa.cache_read(c.k_pages, c.v_pages, c.block_table, cu_of([n]), n, **c.scales)
    ref = P.dequantise(codes, scale)
    np.testing.assert_array_equal(f64(k), ref)
    np.testing.assert_array_equal(f64(v), ref[::-1])


def test_every_code_is_widened_exactly(fa):
    """All 256 bytes as codes: the two NaN codes read as +-480 times the scale
    (no write makes them), every other one exactly."""
    D = 64
    c = Cache([16], 1, D, 16, True, spare=0)
    codes = np.arange(1024, dtype=np.int64).astype(np.uint8).reshape(1, 1, 16, D)
    c.host["k"], c.host["v"] = torch.from_numpy(codes), torch.from_numpy(codes[..., ::-1].copy())
    for e in (-110, -3, 0, 7, 8, 119):
        for s in c.scale_host.values():
            s.fill_(e + 127)
        c.upload()
        k, v = fa.cache_read(c.k_pages, c.v_pages, c.block_table, cu_of([16]), 16, **c.scales)
        ref = P.dequantise(codes[0, 0], np.full(16, e + 127, dtype=np.uint8))
        fine = np.isfinite(ref)
        np.testing.assert_array_equal(f64(k)[:, 0][fine], ref[fine])
        np.testing.assert_array_equal(f64(v)[:, 0][:, ::-1][fine], ref[fine])


def test_padded_entries_are_not_written(fa):
    """A batch entry without a sequence (length 0, or shorter than the new
    tokens): its tokens at negative positions go nowhere, the others are
    written."""
    c = Cache([0, 2, 30], 2, 64, 16, False)
    before = c.raw()
    x = randn((3, 4, 2, 64), 1).cuda()
    fa.cache_write(x, x, c.k_pages, c.v_pages, c.block_table, c.seq_lens)
    clean(fa)
    want = [t.clone() for t in before]
    for b, n in enumerate(c.lens):
        for t in range(4):
            if n - 4 + t >= 0:
                p, s = P.slot_of(c.table, 16, b, n - 4 + t)
                for w in want:
                    w[p, :, s] = x[b, t].cpu().view(torch.int16)
    for got, w in zip(c.raw(), want):
        assert torch.equal(got, w)


def test_write_reports_and_skips_bad_rows(fa):
    c = Cache([20, 20], 1, 64, 16, False)
    before = c.raw()
    x = randn((2, 1, 1, 64), 1).cuda()
    for page in (-1, c.num_pages):
        t = c.block_table.clone()
        t[:, 1] = page
        fa.cache_write(x, x, c.k_pages, c.v_pages, t, c.seq_lens)
        assert fa.get_device_error() == 1
    fa.cache_write(x, x, c.k_pages, c.v_pages, c.block_table, torch.tensor([33, -4], dtype=torch.int32, device="cuda"))
    assert fa.get_device_error() == 1
    for cu in ([0, 5, 2], [0, 2, 1]):
        fa.cache_write(x[:, 0], x[:, 0], c.k_pages, c.v_pages, c.block_table, c.seq_lens * 0,
                       cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert fa.get_device_error() == 1
    for got, w in zip(c.raw(), before):
        assert torch.equal(got, w)
    clean(fa)


def test_many_sequences(fa):
    """1024 sequences, the most: every path of the row search."""
    r = np.random.default_rng(1)
    new = r.integers(0, 3, 1024).tolist()
    lens = [n + int(m) for n, m in zip(new, r.integers(0, 40, 1024))]
    c = Cache(lens, 1, 64, 16, True, seed=5)
    x = randn((sum(new), 1, 64), 2)
    fa.cache_write(x.cuda(), x.cuda(), c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu_of(new),
                   **c.scales)
    clean(fa)
    codes, scale = P.quantise(f64(x))
    value = P.dequantise(codes, scale)
    first, at = 0, 0
    for b, n in enumerate(new):
        first += lens[b]
        c.value["k"][first - n:first] = value[at:at + n]
        c.value["v"][first - n:first] = value[at:at + n]
        at += n
    k, v = fa.cache_read(c.k_pages, c.v_pages, c.block_table, cu_of(lens), sum(lens), **c.scales)
    np.testing.assert_array_equal(f64(k), c.value["k"])
    np.testing.assert_array_equal(f64(v), c.value["v"])
    attend(fa, c, new, 2, True, max_q=2)


# ------------------------------------------------------ as they are used --

def test_serving_loop(fa):
    """Prompts in chunks, then single tokens: rope, write, attend, through a
    quantised cache; the last step is captured into a graph and replayed on
    other values, beside a second graph with a workspace of its own."""
    D, Hq, Hkv, page, B = 128, 8, 2, 16, 3
    prompt = [50, 17, 90]
    steps = [(n, prompt) for n in [None]] + [(1, [p + 1 + i for p in prompt]) for i in range(3)]
    c = Cache([0] * B, Hkv, D, page, True, spare=24, cols=8, junk=0.0)
    c.block_table.copy_(torch.arange(24, dtype=torch.int32, device="cuda").view(3, 8))
    c.table[:] = c.block_table.cpu().numpy()
    hist = {"k": [np.zeros((0, Hkv, D))] * B, "v": [np.zeros((0, Hkv, D))] * B}
    sections = [24, 20, 20]

    def step(q, k, v, pos, lens, cu, ws=None):
        q2, k2 = fa.rope(q, k, pos, sections=sections)
        fa.cache_write(k2, v, c.k_pages, c.v_pages, c.block_table, lens, cu_seqlens=cu, **c.scales)
        o, lse = fa.fwd_paged(q2, c.k_pages, c.v_pages, c.block_table, lens, cu_seqlens=cu, workspace=ws, **c.scales)
        return q2, k2, o, lse

    def inputs(new, lens, seed):
        T = sum(new)
        pos = np.concatenate([np.arange(m - n, m) for n, m in zip(new, lens)])
        pos = torch.tensor(np.stack([pos, pos // 4, pos % 4]), dtype=torch.int32, device="cuda")
        return [randn((T, h, D), seed + i).cuda() for i, h in enumerate((Hq, Hkv, Hkv))] + [pos]

    def check(q2, k2, v, o, lse, new, lens):
        first = 0
        for b, n in enumerate(new):
            for name, x in (("k", k2), ("v", v)):
                hist[name][b] = np.concatenate([hist[name][b][:lens[b] - n],
                                                P.dequantise(*P.quantise(f64(x[first:first + n])))])
            first += n
        c.lens = list(lens)
        c.value = {n: np.concatenate(hist[n]) for n in "kv"}
        check_attention(o, lse, q2, c, new, True, D ** -0.5)

    for i, (n, lens) in enumerate(steps):
        new = [p for p in prompt] if n is None else [1] * B
        q, k, v, pos = inputs(new, lens, 100 * i)
        q2, k2, o, lse = step(q, k, v, pos, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_of(new))
        clean(fa)
        np.testing.assert_allclose(f64(q2), P.rope(f64(q), pos.cpu().numpy(), sections, 10000.0), rtol=2.0 ** -8,
                                   atol=1e-5)
        check(q2, k2, v, o, lse, new, lens)

    # a graph of the step, replayed as the sequences grow
    lens = steps[-1][1]
    dev_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v, pos = inputs([1] * B, lens, 7)
    cu = cu_of([1] * B)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(q, k, v, pos, dev_lens, cu)
    for i in range(3):
        lens = [m + 1 for m in lens]
        new = inputs([1] * B, lens, 1000 + i)
        for to, x in zip((q, k, v, pos), new):
            to.copy_(x)
        dev_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        clean(fa)
        check(out[0], out[1], v, out[2], out[3], [1] * B, lens)


def test_read_back_feeds_dense_attention(fa):
    """cache_read's rows are fwd()'s packed keys and values: one call over
    whole sequences gives what fwd_paged gives."""
    lens = [130, 1, 257]
    c = Cache(lens, 2, 128, 32, True, seed=9)
    q = randn((sum(lens), 4, 128), 4).cuda()
    cu = cu_of(lens)
    k, v = fa.cache_read(c.k_pages, c.v_pages, c.block_table, cu, sum(lens), **c.scales)
    o1, l1 = fa.fwd(q, k, v, causal=True, cu_seqlens=cu)
    o2, l2 = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu, **c.scales)
    clean(fa)
    check_attention(o2, l2, q, c, lens, True, 128 ** -0.5)
    assert (o1.float() - o2.float()).abs().max() <= 2.0 ** -6 * c.value["v"].__abs__().max()
    assert (l1 - l2).abs().max() <= 1e-3


def test_other_stream(fa):
    """Everything on a stream that is not the current one."""
    s = torch.cuda.Stream()
    c = Cache([100, 300], 2, 128, 16, True, seed=6)
    q = randn((2, 1, 8, 128), 4).cuda()
    s.wait_stream(torch.cuda.current_stream())
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, stream=s, **c.scales)
    k, _ = fa.cache_read(c.k_pages, c.v_pages, c.block_table, cu_of(c.lens), 400, stream=s, **c.scales)
    s.synchronize()
    clean(fa)
    check_attention(o.view(2, 8, 128), lse.view(2, 8).t().contiguous(), q.view(2, 8, 128), c, [1, 1], True, 128 ** -0.5)
    np.testing.assert_array_equal(f64(k), c.value["k"])


def test_pages_beyond_32_bit_offsets(fa):
    """A pool of more than 2^31 elements per tensor, its sequence in the last
    pages."""
    num, page, Hkv, D = 33000, 128, 8, 64            # 2.16 G elements
    kp = torch.zeros(num, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.tensor([[num - 1, 0, num - 2]], dtype=torch.int32, device="cuda")
    x = randn((300, Hkv, D), 1)
    y = randn((300, Hkv, D), 2)
    lens, cu = torch.tensor([300], dtype=torch.int32, device="cuda"), cu_of([300])
    fa.cache_write(x.cuda(), y.cuda(), kp, vp, table, lens, cu_seqlens=cu)
    k, v = fa.cache_read(kp, vp, table, cu, 300)
    assert torch.equal(k.cpu(), x) and torch.equal(v.cpu(), y)
    assert torch.equal(kp[num - 2, :, :44].cpu(), x[256:].transpose(0, 1))
    for n in (1, 100):
        q = randn((n, 8, D), 3).cuda()
        o, lse = fa.fwd_paged(q, kp, vp, table, lens, cu_seqlens=cu_of([n]))
        clean(fa)
        c = Cache([0], Hkv, D, page, False)
        c.lens, c.value = [300], {"k": f64(x), "v": f64(y)}
        check_attention(o, lse, q, c, [n], True, D ** -0.5)
