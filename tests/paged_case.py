"""A small paged cache with everything that a test wants to compare: host and
device tensors, and what the cache stands for in fp64."""

import numpy as np
import torch

from oracle import paged as P

from parity import f64


def randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


class Cache:
    """Pages of sequences with `lens` keys, D and page size as given.  Every
    slot that no sequence owns holds `junk` (NaN by default), unused table
    entries are -1, pages are shuffled."""

    def __init__(self, lens, Hkv, D, page, fp8, seed=0, junk=float("nan"), spare=2, cols=None, device="cuda"):
        self.lens, self.Hkv, self.D, self.page, self.fp8, self.device = list(lens), Hkv, D, page, fp8, device
        B = len(self.lens)
        counts = [-(-n // page) for n in self.lens]
        self.num_pages = sum(counts) + spare
        order = torch.randperm(self.num_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        cols = max(1, max(counts)) if cols is None else cols
        self.table = np.full((B, cols), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.num_pages, Hkv, page, D)
        self.host, self.scale_host, self.value = {}, {}, {}
        for i, name in enumerate("kv"):
            rows = randn((sum(self.lens) or 1, Hkv, D), seed * 7 + i + 1)
            if fp8:
                rows = rows * torch.exp2(torch.randint(-3, 4, (rows.shape[0], Hkv, 1),
                                                       generator=torch.Generator().manual_seed(seed + 50 + i)))
                pages = np.full(shape, 0x7F if np.isnan(junk) else 0x38, dtype=np.uint8)
                scale = np.full(shape[:3], 255 if np.isnan(junk) else 127, dtype=np.uint8)
                codes, bytes_ = P.quantise(f64(rows))
                self.value[name] = P.dequantise(codes, bytes_)
            else:
                pages = torch.full(shape, junk, dtype=torch.bfloat16)
                self.value[name] = f64(rows)
            first = 0
            for b, n in enumerate(self.lens):
                for t in range(n):
                    p, s = P.slot_of(self.table, page, b, t)
                    if fp8:
                        pages[p, :, s], scale[p, :, s] = codes[first + t], bytes_[first + t]
                    else:
                        pages[p, :, s] = rows[first + t]
                first += n
            self.host[name] = torch.from_numpy(pages) if fp8 else pages
            self.scale_host[name] = torch.from_numpy(scale) if fp8 else None
        self.upload()

    def upload(self):
        dev = self.device
        view = (lambda t: t.to(dev).view(torch.float8_e4m3fn)) if self.fp8 else (lambda t: t.to(dev))
        self.k_pages, self.v_pages = view(self.host["k"]), view(self.host["v"])
        self.k_scale = self.scale_host["k"].to(dev) if self.fp8 else None
        self.v_scale = self.scale_host["v"].to(dev) if self.fp8 else None
        self.block_table = torch.from_numpy(self.table).to(dev)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=dev)

    @property
    def scales(self):
        return {"k_scale": self.k_scale, "v_scale": self.v_scale}

    def rows(self, name, b):
        first = sum(self.lens[:b])
        return self.value[name][first:first + self.lens[b]]

    def raw(self):
        """The device pages and scales as host integers."""
        out = [t.view(torch.uint8 if self.fp8 else torch.int16).cpu() for t in (self.k_pages, self.v_pages)]
        return out + ([self.k_scale.cpu(), self.v_scale.cpu()] if self.fp8 else [])


def cu_of(new, device="cuda"):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=device)


def check_attention(o, lse, q, cache, new, causal, scale, first=None):
    """o, lse, q packed ([total, Hq, D], [Hq, total]); `first`: the row of each
    sequence's first new token.

    Tolerances.  O: the output is rounded to BF16 (2^-8 relative), and so is
    each weight in the product and in the sum that it is divided by (2^-8 of
    sum |w v| / sum w, twice); 1e-5 for FP32 sums.  LSE: a score is a sum of D
    products in FP32, off by at most D 2^-23 sum |q k| scale, and 2^-21 for
    exponentials and logarithm."""
    first = np.concatenate([[0], np.cumsum(new)]) if first is None else first
    for b, n in enumerate(new):
        if n == 0:
            continue
        i = int(first[b])
        qb, k, v = f64(q[i:i + n]), cache.rows("k", b), cache.rows("v", b)
        o_ref, l_ref, a = P.attention(qb, k, v, causal, scale)
        ob, lb = f64(o[i:i + n]), f64(lse[:, i:i + n])
        assert np.isfinite(ob).all()
        np.testing.assert_array_equal(np.isfinite(lb), np.isfinite(l_ref))
        tol = 2.0 ** -8 * np.abs(o_ref) + 2.0 ** -7 * a + 1e-5
        worst = np.max(np.abs(ob - o_ref) / tol)
        assert worst <= 1.0, (b, worst)
        assert not ob[np.isinf(l_ref).T].any()
        fin = np.isfinite(l_ref)
        if fin.any():
            span = np.abs(qb).sum(-1).max() * np.abs(k).max() * scale
            assert np.max(np.abs(lb[fin] - l_ref[fin])) <= q.shape[-1] * 2.0 ** -23 * span + 2.0 ** -21 * (1 + np.abs(l_ref[fin]).max())
