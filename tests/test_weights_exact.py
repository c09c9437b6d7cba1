"""The criterion of test_weights_exact_gpu.py, without a GPU: it takes what the formula
rounds in FP32, and none of the shorter forms."""

import numpy as np
import pytest

from oracle import paged as P

from weights_exact import SCALE, expected, integers, logsumexp, queries
from parity import f64

F = np.float32
LOG2E = F(1.4426950408889634)


def rounded(x, bits):
    """x with `bits` bits behind the leading one."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(np.ldexp(m, bits + 1)), e - bits - 1)


FORMS = {
    "fp32": lambda s, lse: (F(s * SCALE - lse) * LOG2E).astype(F),
    "fp16 scores": lambda s, lse: (F(s.astype(np.float16).astype(np.float64) * SCALE - lse) * LOG2E).astype(F),
    "10 bits": lambda s, lse: (F(rounded(s, 10) * SCALE - lse) * LOG2E).astype(F),
    "bf16 scores": lambda s, lse: (F(rounded(s, 7) * SCALE - lse) * LOG2E).astype(F),
    "log2 units first": lambda s, lse: (F(s * SCALE * float(LOG2E)) - F(lse) * LOG2E).astype(F),
    "bf16 lse": lambda s, lse: (F(s * SCALE - rounded(np.float64(lse), 7)) * LOG2E).astype(F),
    "fp16 difference": lambda s, lse: (F(s * SCALE - lse).astype(np.float16).astype(F) * LOG2E).astype(F),
}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,live", [(1, 4), (8, 32), (60, 1), (60, 240)])
@pytest.mark.parametrize("form", FORMS)
def test_criterion(form, n, live, D):
    """n tokens of 4 heads over 500 keys, `live` rows of them with an LSE."""
    L, Hq = 500, 4
    k, q = integers((L, 1, D), 8, n + D), f64(queries(n, Hq, D, n))
    sees = P.causal_sees(n, L, True)
    alive = np.zeros(n * Hq, dtype=bool)
    alive[np.random.default_rng(1).permutation(n * Hq)[:live]] = True
    alive = alive.reshape(Hq, n)
    lse = logsumexp(q, k, sees, SCALE, alive)
    want, tol = expected(q, lse, k, sees, SCALE)
    got = np.zeros(L, dtype=F)
    for h in range(Hq):
        s = q[:, h] @ k[:, 0].T
        assert np.array_equal(s, np.round(s)) and np.abs(s).max() < 2 ** 16
        for i in np.flatnonzero(alive[h]):
            w = np.exp2(FORMS[form](s[i], lse[h, i]).astype(np.float64)).astype(F)
            got = np.where(sees[i], (got + np.where(w < 2.0 ** -126, F(0), w)).astype(F), got)
    worst = np.max(np.abs(got - want[0]) / tol[0])
    if form == "fp32":
        assert worst <= 1.0
    elif form == "log2 units first" and live > 32:
        pass        # (hidden by the rounding of a sum of 240 weights)
    else:
        assert worst > 1.5, worst
