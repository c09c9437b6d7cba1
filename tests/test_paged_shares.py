"""The criterion of the shares tests rejects what it is there to reject, and lets the
roundings of the kernels through.  On the CPU, with the oracle alone."""

import numpy as np
import pytest
import torch

from oracle import paged as P

from paged_case import randn
from paged_shares import one_hot_values, shares_cache, worst
from parity import f64

D, HEADS, SCALE = 128, 8, 128 ** -0.5


@pytest.fixture(scope="module", params=[9001, 50001])
def case(request):
    L = request.param
    q = f64(randn((1, HEADS, D), 3))
    k = f64(randn((L, 1, D), 4))
    return q, k, one_hot_values(L, 1, D)


def weights(q, k):
    s = np.einsum("hd,ld->hl", q[0], k[:, 0]) * SCALE
    return np.exp(s - s.max(-1, keepdims=True))


def bf16(x):
    return f64(torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16))


def test_roundings_pass(case):
    q, k, v = case
    w = weights(q, k)
    o = bf16(bf16(w) @ v[:, 0] / bf16(w).sum(-1, keepdims=True))
    assert worst(o[None], q, k, v, False, SCALE, False) <= 1.0
    h = (w * 64).astype(np.float16).astype(np.float64) / 64
    o = bf16(h @ v[:, 0] / w.sum(-1, keepdims=True))
    assert worst(o[None], q, k, v, False, SCALE, True) <= 1.0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", ["values", "keys", "shifted", "twice"])
@pytest.mark.parametrize("at,keys", [(0, 128), (4992, 128), (5003, 59), (8960, 41)])
def test_faults_are_rejected(case, fp8, what, at, keys):
    """A block's values lost, its keys lost with them (a part that is not joined),
    the next block's values in their place, or a part joined twice."""
    q, k, v = case
    w = weights(q, k)
    lost = slice(at, at + keys)
    wv, ws, bad = w.copy(), w.copy(), v.copy()
    if what in ("values", "keys"):
        wv[:, lost] = 0
    if what == "keys":
        ws[:, lost] = 0
    if what == "shifted":      # from two stretches on: a neighbour's may be the same column
        step = 2 * -(-len(k) // D)
        bad[lost] = np.roll(v, -step, axis=0)[lost]
    if what == "twice":
        wv[:, lost] *= 2
        ws[:, lost] *= 2
    o = bf16(wv @ bad[:, 0] / ws.sum(-1, keepdims=True))
    assert worst(o[None], q, k, v, False, SCALE, fp8) > 1.5


@pytest.mark.parametrize("fp8", [False, True])
def test_the_cache_holds_what_it_says(fp8):
    c = shares_cache([300, 5], 2, 64, 32, fp8, seed=1, device="cpu")
    for b, n in enumerate(c.lens):
        rows = P.gather(c.host["v"].numpy() if fp8 else c.host["v"].view(torch.int16).numpy(), c.table, b, n)
        got = P.dequantise(rows, P.gather(c.scale_host["v"].numpy(), c.table, b, n)) if fp8 else \
            f64(torch.from_numpy(rows).view(torch.bfloat16))
        np.testing.assert_array_equal(got, c.rows("v", b))
        assert (got.sum(-1) == 1).all() and (got.sum(0) > 0).sum() >= min(n, 60)
