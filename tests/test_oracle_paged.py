"""The plain forms that the paged-cache tests compare with, on the CPU: against
torch's E4M3, closed forms and differences."""

import numpy as np
import pytest
import torch

from oracle import paged as P


def test_e4m3_codes_match_torch(rng):
    y = np.concatenate([rng.normal(size=5000) * 10.0 ** rng.uniform(-4, 2, 5000), P.e4m3_grid(), -P.e4m3_grid(),
                        (P.e4m3_grid()[1:] + P.e4m3_grid()[:-1]) / 2])       # every tie
    y = np.clip(y.astype(np.float32), -448, 448)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(P.e4m3_codes(y.astype(np.float64)), want.view(torch.uint8).numpy())
    np.testing.assert_array_equal(P.e4m3_values(want.view(torch.uint8).numpy()), want.double().numpy())


@pytest.mark.parametrize("amax,e", [(448.0, 0), (450.0, 1), (1.75, -8), (1.7500001, -7), (0.0, -110), (1e-39, -110),
                                    (3.0e38, 119), (448.0 * 2.0 ** 119, 119)])
def test_scale_exponent(amax, e):
    codes, s = P.quantise(np.array([[amax, -amax / 2]]))
    assert s[0] == e + 127
    assert np.all(np.abs(P.e4m3_values(codes)) <= 448)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_rows_that_are_not_finite_stand_for_nan(bad):
    codes, s = P.quantise(np.array([[1.0, bad], [1.0, 2.0]]))
    assert s[0] == 255 and not codes[0].any()
    back = P.dequantise(codes, s)
    assert np.isnan(back[0]).all() and np.array_equal(back[1], [1.0, 2.0])


def test_quantisation_error_is_half_a_step(rng):
    x = rng.normal(size=(200, 64))
    codes, s = P.quantise(x)
    step = 2.0 ** (s.astype(float) - 127)[:, None]
    assert np.all(np.abs(P.dequantise(codes, s) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * step))


def test_attention_closed_forms(rng):
    v = rng.normal(size=(5, 1, 8))
    q, k = np.zeros((3, 2, 8)), rng.normal(size=(5, 1, 8))
    o, lse, _ = P.attention(q, k, v, True, 0.3)          # rows see 3, 4, 5 keys, all alike
    for i in range(3):
        np.testing.assert_allclose(o[i, 0], v[:3 + i, 0].mean(0))
        np.testing.assert_allclose(lse[:, i], np.log(3 + i))
    o, lse, _ = P.attention(q, k[:1], v[:1], True, 0.3)  # two rows see nothing
    assert not o[:2].any() and np.all(lse[:, :2] == -np.inf)
    np.testing.assert_allclose(o[2, 1], v[0, 0])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("restart", [False, True])
def test_rope_gradient_is_the_inverse_rotation(rng, interleaved, restart):
    """Against differences: the gradient of <rope(x), w> is rope(w, inverse)."""
    x, w = rng.normal(size=(2, 1, 12)), rng.normal(size=(2, 1, 12))
    pos = np.array([[3, 70000], [5, -2]])
    kw = dict(sections=[2, 3], base=100.0, restart=restart, interleaved=interleaved)
    g = P.rope(w, pos, inverse=True, **kw)
    for i in range(12):
        d = np.zeros_like(x)
        d[:, :, i] = 1e-6
        up, down = (P.rope(x + s * d, pos, **kw) for s in (1, -1))
        diff = ((up - down) * w).sum(-1) / 2e-6
        np.testing.assert_allclose(diff[:, 0], g[:, 0, i], atol=1e-8)
    np.testing.assert_allclose(P.rope(P.rope(x, pos, **kw), pos, inverse=True, **kw), x, atol=1e-12)
    np.testing.assert_array_equal(P.rope(x, pos, **kw)[..., 10:], x[..., 10:])      # not rotated
