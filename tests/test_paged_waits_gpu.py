"""The attention kernels' waits last a key block or so, however long sequences are:
calls whose segments take many times the limit of a wait end in time, without a
give-up."""

import math

import numpy as np
import pytest
import torch

from oracle import paged as P

from paged_waits import Repeated
from parity import f64

pytestmark = pytest.mark.gpu

LIMIT_NS = 2_000_000
REPEAT = 8192            # a million keys, 10 ms for a chunk's rows


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,B", [(30, 760), (1, 152)])
def test_long_segments(fa, new, B, fp8):
    """30 tokens of 4 heads fill one tile of a pair: the other tile's warps have
    nothing to do for five segments' time."""
    r = Repeated(fa, B, new, fp8, REPEAT)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in "se")
    start.record()
    status = r.call(LIMIT_NS)
    end.record()
    end.synchronize()
    assert status == 0
    if new > 1:
        assert start.elapsed_time(end) * 1e6 > 5 * 2 * LIMIT_NS        # five segments, each twice the limit or more
    # the same weights on each repetition of a key: O as over one page, LSE log(repeat) more
    k, v = r.c.rows("k", 0), r.c.rows("v", 0)
    for b in (0, 1, B // 2, B - 1):
        q = f64(r.q[b])
        o_ref, l_ref, a = P.attention(q, k, v, False, r.scale)
        # as for other calls, and FP32 sums over REPEAT blocks, eight products each
        tol = 2.0 ** -8 * np.abs(o_ref) + (2.0 ** -7 + 8 * REPEAT * 2.0 ** -23) * a + 1e-5
        assert np.all(np.abs(f64(r.o[b]) - o_ref) <= tol)
        span = np.abs(q).sum(-1).max() * np.abs(k).max() * r.scale
        err = np.abs(f64(r.lse[b]) - l_ref - math.log(REPEAT)).max()
        assert err <= r.D * 2.0 ** -23 * span + REPEAT * 2.0 ** -23 + 2.0 ** -18
