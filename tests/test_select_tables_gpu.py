"""Selections under block tables that are wider than the longest sequence, as a serving
program has one width for all its batches."""

import pytest

from test_evict_gpu import Sums

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


@pytest.mark.parametrize("width", [4096, 65536, 1 << 20])
@pytest.mark.parametrize("lens,Hkv", [([1], 1), ([0, 700, 41], 2), ([5000] * 20, 8), ([300] * 48, 8)])
def test_wide_tables(fa, lens, Hkv, width):
    """A single head, a few, as many as SMs, and more than two blocks an SM."""
    s = Sums(lens, Hkv, 64, seed=len(lens), cols=max(-(-max(lens) // 64), width // 64))
    for keep, first, recent in ((40, 3, 7), (600, 0, 0)):
        s.check(fa, keep, first, recent)
