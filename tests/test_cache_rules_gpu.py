"""Cache writes and read-back where one sequence of a batch breaks the rules of
offsets and lengths: all of its rows are skipped, none in part, the call reports
it, and the other sequences are served."""

import pytest
import torch

from paged_case import Cache, randn
from oracle import paged as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def written(c, before, x, tokens):
    """`before` with row i of x at (sequence, position) tokens[i], as BF16 bits."""
    want = [t.clone() for t in before]
    for i, (b, pos) in tokens.items():
        p, s = P.slot_of(c.table, c.page, b, pos)
        for w in want:
            w[p, :, s] = x[i].cpu().view(torch.int16)
    return want


@pytest.mark.parametrize("length", [33, 35, 2 ** 31 - 1, -1, -2 ** 31])
@pytest.mark.parametrize("dense", [False, True])
def test_a_length_out_of_range_writes_nothing(fa, dense, length):
    """Lengths that leave some of the new tokens within the table, too."""
    c = Cache([32, 20, 32], 1, 64, 16, False, seed=1)             # the table holds 32 tokens a sequence
    before = c.raw()
    x = randn((12, 1, 64), 2).cuda()
    y = x.view(3, 4, 1, 64) if dense else x
    fa.cache_write(y, y, c.k_pages, c.v_pages, c.block_table, ints(length, 20, 30),
                   cu_seqlens=None if dense else ints(0, 4, 8, 12))
    assert fa.get_device_error() == 1
    tokens = {4 + i: (1, 16 + i) for i in range(4)}
    tokens.update({8 + i: (2, 26 + i) for i in range(4)})
    for got, w in zip(c.raw(), written(c, before, x, tokens)):
        assert torch.equal(got, w)


def test_offsets_behind_the_rows_write_nothing(fa):
    c = Cache([20, 20], 1, 64, 16, False, seed=1)
    before = c.raw()
    x = randn((6, 1, 64), 2).cuda()
    fa.cache_write(x, x, c.k_pages, c.v_pages, c.block_table, ints(20, 20), cu_seqlens=ints(0, 2, 9))
    assert fa.get_device_error() == 1
    for got, w in zip(c.raw(), written(c, before, x, {0: (0, 18), 1: (0, 19)})):
        assert torch.equal(got, w)


def test_a_first_offset_that_is_not_zero_writes_nothing(fa):
    c = Cache([20, 20], 1, 64, 16, False, seed=1)
    before = c.raw()
    x = randn((6, 1, 64), 2).cuda()
    fa.cache_write(x, x, c.k_pages, c.v_pages, c.block_table, ints(20, 20), cu_seqlens=ints(1, 3, 6))
    assert fa.get_device_error() == 1
    for got, w in zip(c.raw(), written(c, before, x, {3 + i: (1, 17 + i) for i in range(3)})):
        assert torch.equal(got, w)


@pytest.mark.parametrize("cu", [(0, 10, 45, 50), (0, 10, 20, 60)])
def test_read_back_leaves_the_rows_of_a_bad_sequence(fa, cu):
    """Longer than the table, or behind the rows there are."""
    c = Cache([32, 32, 32], 1, 64, 16, False, seed=3)
    k, v = (torch.full((52, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    fa.cache_read(c.k_pages, c.v_pages, c.block_table, ints(*cu), 52, k_out=k, v_out=v)
    assert fa.get_device_error() == 1
    for name, got in (("k", k), ("v", v)):
        want = torch.full((52, 1, 64), 7.0, dtype=torch.float64)
        for b in range(3):
            n = cu[b + 1] - cu[b]
            if n <= 32 and cu[b + 1] <= 52:
                want[cu[b]:cu[b + 1]] = torch.from_numpy(c.rows(name, b)[:n])
        assert torch.equal(got.cpu().double(), want)
    assert fa.get_device_error() == 0
