"""Sums of weights over E4M3 pages whose queries, keys and scale are far from one, but
whose scores are not: what test_paged_scales_gpu.py asks of the attention."""

import pytest
import torch

from paged_case import Cache, randn
from test_paged_scales_gpu import PAIRS, shift_keys
from weights_case import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


# keys next to the largest, and queries next to the least and the largest
FAR = PAIRS + [(-122, 118), (-60, 118), (115, -95)]


def weigh(fa, D, new, Hq, q_exp, k_exp):
    c = Cache([300, 140, max(new, 5)], 1, D, 32, True, seed=D + new)
    shift_keys(c, k_exp)
    q = torch.ldexp(randn((3 * new, Hq, D), 5).double(), torch.tensor(q_exp)).to(torch.bfloat16)
    check(fa, c, [new] * 3, Hq, q=q, scale=2.0 ** (-q_exp - k_exp - 4))


def largest_keys(fa, D, new, scale, score):
    """Keys of all of BF16's range, alike along D; the largest score is about `score`."""
    c = Cache([90], 1, D, 16, True, seed=1)
    g = torch.Generator().manual_seed(2)
    own = c.scale_host["k"] != 255
    c.host["k"][:] = 0x7E                                              # 448
    e = torch.randint(112, 120, own.shape, generator=g)
    c.scale_host["k"] = torch.where(own, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    for t in range(90):
        c.value["k"][t] = 448 * 2.0 ** float(e[c.table[0, t // 16], 0, t % 16])
    c.upload()
    size = score / (D * 448 * 2.0 ** 119 * scale)
    q = (torch.rand(new, 4, 1, generator=g) + 0.5).expand(new, 4, D).double() * size
    check(fa, c, [new], 4, q=q.to(torch.bfloat16).contiguous(), scale=scale)


LARGEST = [(128, 2.0 ** -113, 3.5), (64, 2.0 ** -112, 3.5), (128, 1.3 * 2.0 ** -126, 3.5), (64, 1.3 * 2.0 ** -126, 40.0),
           (128, 1.7 * 2.0 ** -122, 40.0)]


@pytest.mark.parametrize("q_exp,k_exp", FAR)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,Hq", [(1, 4), (4, 4), (7, 4)])
def test_few_rows(fa, new, Hq, D, q_exp, k_exp):
    weigh(fa, D, new, Hq, q_exp, k_exp)


@pytest.mark.parametrize("D,scale,score", LARGEST)
@pytest.mark.parametrize("new", [1, 4, 8])
def test_few_rows_over_the_largest_keys(fa, new, D, scale, score):
    largest_keys(fa, D, new, scale, score)


@pytest.mark.parametrize("q_exp,k_exp", FAR)
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows(fa, D, q_exp, k_exp):
    weigh(fa, D, 50, 4, q_exp, k_exp)


@pytest.mark.parametrize("D,scale,score", LARGEST)
@pytest.mark.parametrize("new", [9, 50])
def test_many_rows_over_the_largest_keys(fa, new, D, scale, score):
    largest_keys(fa, D, new, scale, score)
