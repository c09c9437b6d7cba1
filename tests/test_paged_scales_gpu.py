"""Attention over E4M3 pages whose queries, keys and scale are far from one, but
their product is not: the powers of two that the kernels take out of each cancel."""

import pytest
import torch

from paged_case import Cache, check_attention, cu_of, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


def shift_keys(c, e):
    """The cache's keys times 2^e: their scale bytes alone."""
    own = c.scale_host["k"] != 255
    byte = c.scale_host["k"].int() + e
    assert ((byte >= 17) & (byte <= 246))[own].all()
    c.scale_host["k"] = torch.where(own, byte, torch.full_like(byte, 255)).to(torch.uint8)
    c.value["k"] = c.value["k"] * 2.0 ** e
    c.upload()


def attend(fa, D, new, Hq, q_exp, k_exp, scale):
    lens = [300, 140, max(new, 5)]
    c = Cache(lens, 1, D, 32, True, seed=D + new)
    shift_keys(c, k_exp)
    q = torch.ldexp(randn((3 * new, Hq, D), 5).double(), torch.tensor(q_exp)).to(torch.bfloat16).cuda()
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu_of([new] * 3), max_q=new,
                          scale=scale, **c.scales)
    assert fa.get_device_error() == 0
    check_attention(o, lse, q, c, [new] * 3, True, scale)
    return lse


# queries of 2^q_exp and keys of 2^k_exp with a scale that brings the scores back
PAIRS = [(-60, -60), (-120, 0), (-126, 20), (100, -95), (-100, 100), (60, 60), (110, -95), (-20, -95)]


@pytest.mark.parametrize("q_exp,k_exp", PAIRS)
@pytest.mark.parametrize("D", [64, 128])
def test_chunk_scores_of_ordinary_size(fa, D, q_exp, k_exp):
    lse = attend(fa, D, 50, 4, q_exp, k_exp, 2.0 ** (-q_exp - k_exp - 4))
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("D", [64, 128])
def test_chunk_scores_near_zero(fa, D):
    """Scores of 2^-13 at a scale of 2^100: every key counts alike."""
    attend(fa, D, 50, 4, -60, -60, 2.0 ** 100)


@pytest.mark.parametrize("D", [64, 128])
def test_chunk_rows_of_unlike_size(fa, D):
    """Rows of one tile, 2^-120 to 2^120 and zero, the scale for the middle."""
    c = Cache([200], 1, D, 32, True, seed=3)
    q = randn((50, 4, D), 5).double()
    q[0::4] *= 2.0 ** 70
    q[1::4] *= 2.0 ** -90
    q[2::4] = 0
    q = q.to(torch.bfloat16).cuda()
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu_of([50]), max_q=50,
                          scale=2.0 ** -74, **c.scales)
    assert fa.get_device_error() == 0
    check_attention(o, lse, q, c, [50], True, 2.0 ** -74)


@pytest.mark.parametrize("q_exp,k_exp", PAIRS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 4])
def test_single_tokens_scores_of_ordinary_size(fa, new, D, q_exp, k_exp):
    lse = attend(fa, D, new, 4, q_exp, k_exp, 2.0 ** (-q_exp - k_exp - 4))
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("new", [1, 4, 50])
@pytest.mark.parametrize("D,scale", [(128, 2.0 ** -113), (64, 2.0 ** -112), (128, 1.3 * 2.0 ** -126)])
def test_the_largest_keys_with_a_small_scale(fa, new, D, scale):
    """Keys of all of BF16's range, alike along D, so that the scores of an FP16
    row and a row of codes are the largest there are, and the factor that brings
    them back is below the normal numbers."""
    c = Cache([90], 1, D, 16, True, seed=1)
    g = torch.Generator().manual_seed(2)
    own = c.scale_host["k"] != 255
    c.host["k"][:] = 0x7E                                              # 448
    e = torch.randint(112, 120, own.shape, generator=g)
    c.scale_host["k"] = torch.where(own, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    for t in range(90):
        c.value["k"][t] = 448 * 2.0 ** float(e[c.table[0, t // 16], 0, t % 16])
    c.upload()
    size = 3.5 / (D * 448 * 2.0 ** 119 * scale)                        # the largest score is about 3.5
    q = (torch.rand(new, 4, 1, generator=g) + 0.5).expand(new, 4, D).double() * size
    q = q.to(torch.bfloat16).contiguous().cuda()
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu_of([new]), max_q=new,
                          scale=scale, **c.scales)
    assert fa.get_device_error() == 0
    check_attention(o, lse, q, c, [new], True, scale)
