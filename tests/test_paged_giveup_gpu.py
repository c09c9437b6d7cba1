"""Attention kernels whose waits give up end, report it and leave the GPU as it was:
the same call with the usual limit gives what it gave before."""

import pytest
import torch

from paged_waits import Repeated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


def test_chunk_kernel_gives_up(fa):
    """E4M3: before a segment's first tile all of its scales are looked at, which
    over two million keys takes many times 20 us."""
    r = Repeated(fa, 152, 30, True, 16384)
    assert r.call(2 * 10 ** 9) == 0
    o, lse = r.o.clone(), r.lse.clone()
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
    for _ in range(3):
        assert r.call(20_000) == fa.binding.FA_ERR_TIMEOUT
        assert r.call(2 * 10 ** 9) == 0
        assert torch.equal(r.o, o) and torch.equal(r.lse, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_kernel_gives_up(fa, fp8):
    """The warp that looks pages up is done with a batch in less time than the
    others take for it."""
    r = Repeated(fa, 152, 1, fp8, 512)
    assert r.call(2 * 10 ** 9) == 0
    o, lse = r.o.clone(), r.lse.clone()
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
    for _ in range(3):
        assert r.call(1) == fa.binding.FA_ERR_TIMEOUT
        assert r.call(2 * 10 ** 9) == 0
        assert torch.equal(r.o, o) and torch.equal(r.lse, lse)
