"""Rows that see no key, next to rows of the same tile that do: O = 0 and
LSE = -inf, also where the values hold NaN and infinities."""

import pytest
import torch

from paged_case import Cache, check_attention, cu_of, randn
from oracle import paged as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,keys,Hq", [(4, 2, 4), (2, 1, 16), (60, 3, 4), (60, 59, 2), (700, 600, 8), (1500, 900, 2)])
def test_rows_without_keys_beside_values_that_are_not_finite(fa, new, keys, Hq, D, fp8):
    c = Cache([keys, 40], 1, D, 16, fp8, seed=new)
    for t in (0, keys - 1):
        p, s = P.slot_of(c.table, c.page, 0, t)
        if fp8:
            c.host["v"][p, :, s], c.scale_host["v"][p, :, s] = 0, 255
        else:
            c.host["v"][p, :, s] = float("inf") if t else float("nan")
    c.upload()
    news = [new, 1]
    q = randn((sum(news), Hq, D), 2).cuda()
    o, lse = fa.fwd_paged(q, c.k_pages, c.v_pages, c.block_table, c.seq_lens, cu_seqlens=cu_of(news), max_q=new, **c.scales)
    assert fa.get_device_error() == 0
    none = new - keys
    assert not o[:none].any() and not torch.isnan(o[:none].float()).any()
    assert (lse[:, :none] == -float("inf")).all() and torch.isfinite(lse[:, none:]).all()
    assert torch.isnan(o[none:new].float()).all()                 # token 0 is NaN, and all of these see it
    c.lens, c.value = c.lens[1:], {n: v[keys:] for n, v in c.value.items()}
    check_attention(o[new:], lse[:, new:], q[new:], c, [1], True, D ** -0.5)
