"""Long, split and ragged sequences over values that show each share of the weights:
no block of keys is lost, misplaced or joined twice."""

import numpy as np
import pytest

from paged_case import cu_of, randn
from paged_shares import check_shares, shares_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


def attend(fa, c, new, Hq, causal=True, seed=3):
    q = randn((sum(new), Hq, c.D), seed).cuda()
    o, _ = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, causal=causal, cu_seqlens=cu_of(new),
                        max_q=max(new), **c.scales)
    assert fa.get_device_error() == 0
    check_shares(o, q, c, new, causal, c.D ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L,page,new,Hq", [(9001, 128, 1, 8), (9001, 16, 70, 8), (50001, 16, 1, 8), (50001, 64, 20, 8),
                                           (4097, 1024, 130, 2)])
def test_one_sequence_over_all_blocks(fa, L, page, new, Hq, D, fp8):
    attend(fa, shares_cache([L], 1, D, page, fp8, seed=L + new), [new], Hq)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("most", [1, 2, 90])
def test_ragged_sequences(fa, most, causal, fp8):
    """Units of unlike length, cut where the stretches' borders fall."""
    r = np.random.default_rng(most)
    new = r.integers(1, most + 1, 24).tolist()
    lens = [n + int(m) for n, m in zip(new, np.exp(r.uniform(0, np.log(5000), 24)))]
    attend(fa, shares_cache(lens, 2, 128, 32, fp8, seed=most), new, 8, causal)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,L", [(1, 1000), (60, 700)])
def test_as_many_units_as_blocks(fa, new, L, fp8):
    """Whole rounds of the chunk kernel, and a line that is cut near units' ends."""
    B = 76
    attend(fa, shares_cache([L] * B, 2, 64, 64, fp8, seed=new), [new] * B, 8)
