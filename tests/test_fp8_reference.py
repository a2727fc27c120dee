"""Pins of the plain 64-bit forms (tests/fp8_reference.py): hand-worked values,
torch's own e4m3 conversion, and the norm's gradient against differences."""
import numpy as np
import pytest
import torch

import fp8_reference as ref


def test_exponent_by_hand():
    # 448 fits as it is; the next value up needs twice the scale; 3.5 = 448 / 128
    assert ref.least_exponent(448.0) == 0
    assert ref.least_exponent(np.nextafter(448.0, 1e9)) == 1
    assert ref.least_exponent(3.5) == -7
    assert ref.least_exponent(0.0) == 0
    assert ref.least_exponent(1e-45) == -127


def test_rounding_by_hand():
    # mantissa step at [16, 32) is 2: 17 and 19 are ties, to even multiples
    got = ref.round_e4m3([17.0, 19.0, 18.9, 448.0, 2.0 ** -10, 3 * 2.0 ** -10, np.inf, np.nan])
    assert np.array_equal(got[:6], [16.0, 20.0, 18.0, 448.0, 0.0, 2.0 ** -8])
    assert np.isnan(got[6:]).all()


def test_rounding_matches_torch():
    x = torch.linspace(-448, 448, 100001, dtype=torch.float32)
    x = torch.cat([x, x * 2.0 ** -9, x * 2.0 ** -15])
    want = x.to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.round_e4m3(x.double().numpy()), want)


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_uses_its_range(rows):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((200, 300)) * np.exp(rng.standard_normal((200, 1)) * 8)
    v, e = ref.quantize(x, rows)
    assert np.abs(v).max() <= 448
    # half a step of a normal value is 2^-4 of it; below 2^-6 half a step is 2^-10
    scale = ref.dequantize(np.ones_like(v), e, rows)
    assert (np.abs(v * scale - x) <= np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10)).all()
    if rows == 1:                       # no smaller scale would have done
        top = np.abs(x[:, :128]).max(axis=1)
        assert (top > 448 * 2.0 ** (e[:, 0] - 1.0)).all()


@pytest.mark.parametrize("residual_grad", [False, True])
def test_norm_gradient_against_differences(residual_grad):
    rng = np.random.default_rng(5)
    h, w, dy = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7))
    dh = rng.standard_normal((3, 7)) if residual_grad else None

    def loss(h, w):
        y, _ = ref.norm(h, w, 1e-6)
        return (y * dy).sum() + (0 if dh is None else (h * dh).sum())

    dx, dw = ref.norm_backward(dy, h, ref.norm(h, w, 1e-6)[1], w, dh)
    # central differences of step t are off by O(t^2) + rounding / t
    t = 1e-5
    for i in np.ndindex(*h.shape):
        d = np.zeros_like(h)
        d[i] = t
        assert abs((loss(h + d, w) - loss(h - d, w)) / (2 * t) - dx[i]) < 1e-7
    for i in range(7):
        d = np.zeros_like(w)
        d[i] = t
        assert abs((loss(h, w + d) - loss(h, w - d)) / (2 * t) - dw[i]) < 1e-7
