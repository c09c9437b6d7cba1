"""Calls of the paged attention with a wait limit of the test's, over sequences of
one page over and over."""

import torch

from paged_case import Cache, randn


class Repeated:
    """B sequences of `repeat` times the same page of 128 keys, `new` tokens each,
    4 heads on one key/value head, D = 64, no mask."""

    Hq, D = 4, 64
    scale = D ** -0.5

    def __init__(self, fa, B, new, fp8, repeat):
        self.fa, self.B, self.new, self.repeat = fa, B, new, repeat
        self.c = Cache([128], 1, self.D, 128, fp8, seed=1)
        self.table = self.c.block_table[:, :1].expand(B, repeat).contiguous()
        self.lens = torch.full((B,), 128 * repeat, dtype=torch.int32, device="cuda")
        self.q = randn((B, new, self.Hq, self.D), 2).cuda()
        self.o, self.lse = torch.empty_like(self.q), torch.empty(B, self.Hq, new, device="cuda")
        self.need = fa.fwd_paged_workspace_size(B, self.Hq, 1, new, self.D)
        self.ws = torch.empty(self.need, dtype=torch.uint8, device="cuda")

    def call(self, limit_ns):
        """The status of the device after the call."""
        adr = lambda t: None if t is None else t.data_ptr()
        c = self.c
        self.o.fill_(float("nan"))
        self.lse.fill_(float("nan"))
        st = self.fa.load_library().fa_diag_fwd_paged(
            adr(self.q), adr(c.k_pages), adr(c.v_pages), adr(c.k_scale), adr(c.v_scale), adr(self.o), adr(self.lse), self.B,
            self.Hq, 1, self.new, self.D, c.num_pages, 128, self.repeat, 0, self.scale, adr(self.table), adr(self.lens), None,
            0, adr(self.ws), self.need, limit_ns, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        return self.fa.get_device_error()
