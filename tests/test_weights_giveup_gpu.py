"""Kernels of cache_weights whose waits give up end, report it and leave the GPU as it
was: the same call gives what it gave before.  A barrier of each thread block (or warp)
waits for bytes that nobody brings; whoever waits for it gives up after a millisecond,
wherever the others are then."""

import pytest
import torch

from paged_case import Cache, randn

pytestmark = pytest.mark.gpu

LIMIT_NS = 10 ** 6


@pytest.fixture(scope="module")
def fa():
    import exact_attention_78_gb300 as fa_mod
    fa_mod.load_library(build_if_missing=True)
    return fa_mod


class Call:
    """B sequences of `repeat` times the same page of 128 keys, n tokens each, 4 heads on one
    key/value head, no mask; with decay 0 the repeated slots' sums are all the same."""

    def __init__(self, fa, B, n, D, fp8, repeat):
        self.fa, self.shape = fa, (B, 4, 1, n, D)
        self.c = Cache([128], 1, D, 128, fp8, seed=1)
        # each sequence has its own page of sums behind the keys' ones: pages are not shared
        self.k = self.c.k_pages[self.c.table[0, 0]].unsqueeze(0).expand(B * repeat, 1, 128, D).contiguous()
        self.ks = None if not fp8 else self.c.k_scale[self.c.table[0, 0]].unsqueeze(0).expand(B * repeat, 1, 128).contiguous()
        self.table = torch.arange(B * repeat, dtype=torch.int32, device="cuda").view(B, repeat)
        self.lens = torch.full((B,), 128 * repeat, dtype=torch.int32, device="cuda")
        self.q = randn((B, n, 4, D), 2).cuda()
        self.lse = torch.full((B, 4, n), 3.0, device="cuda")
        self.sums = torch.empty(B * repeat, 1, 128, device="cuda")

    def __call__(self, held=-1):
        """The status of the device after the call."""
        adr = lambda t: None if t is None else t.data_ptr()
        self.sums.fill_(float("nan"))
        st = self.fa.load_library().fa_diag_cache_weights(
            adr(self.q), adr(self.lse), adr(self.k), adr(self.ks), adr(self.sums), *self.shape, self.k.shape[0], 128,
            self.table.shape[1], 0, self.shape[-1] ** -0.5, 0.0, adr(self.table), adr(self.lens), None, 0, LIMIT_NS, held,
            torch.cuda.current_stream().cuda_stream)
        assert st == 0
        return self.fa.get_device_error()


def gives_up(fa, call, barriers):
    assert call() == 0
    want = call.sums.clone()
    assert torch.isfinite(want).all()
    for held in barriers:
        assert call(held) == fa.binding.FA_ERR_TIMEOUT, held
        assert call() == 0
        assert torch.equal(call.sums, want), held


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 8])
def test_few_rows(fa, n, D, fp8):
    """The first stages of each warp's ring, reached while later ones are on their way."""
    gives_up(fa, Call(fa, 64, n, D, fp8, 24), [0, 1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,barriers", [(64, 22), (128, 18)])
def test_many_rows(fa, D, barriers, fp8):
    """Every barrier that a role waits for tile by tile; a block has five units of two
    tiles of rows, so that each comes round a second time."""
    gives_up(fa, Call(fa, 64, 64, D, fp8, 24), range(barriers))
