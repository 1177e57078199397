"""The 8-bit oracle against closed forms, and its gradient against differences."""
import numpy as np
import pytest

from oracle import int8 as o8


def test_codes_are_nearest_with_ties_to_even():
    x = np.array([[254.0, 1.0, 3.0, 5.0, -1.0, -3.0, 2.0, 0.0]])    # 127 x / 254 = x / 2
    codes, scale = o8.quantize_rows(x)
    assert codes.tolist() == [[127, 0, 2, 2, 0, -2, 1, 0]]
    assert scale[0] == np.float32(2.0)


def test_zero_and_non_finite_rows():
    x = np.array([[0.0, 0.0], [1.0, np.inf], [np.nan, 2.0], [-4.0, 4.0]])
    codes, scale = o8.quantize_rows(x)
    assert codes.tolist() == [[0, 0], [0, 0], [0, 0], [-127, 127]]
    assert scale[0] == 0 and np.isnan(scale[1]) and np.isnan(scale[2])
    assert scale[3] == np.float32(4.0) / np.float32(127.0)


@pytest.mark.parametrize("block", [0, 64])
def test_values_are_within_half_a_step(block):
    x = np.random.default_rng(3).standard_normal((5, 192)).astype(np.float32)
    codes, scale = o8.quantize_rows(x, block)
    step = np.repeat(scale, 64, 1) if block else np.repeat(scale[:, None], 192, 1)
    # half a step, the scale's rounding at code 127
    assert np.all(np.abs(o8.values(codes, scale) - x) <= step * (0.5 + 127 * 2.0 ** -24))


def test_gating_gradient_against_differences():
    g = np.random.default_rng(4)
    G, U, dH = (g.standard_normal(40) for _ in range(3))
    dG, dU = o8.silu_mul_grad(dH, G, U)
    h = 1e-6
    num_G = dH * (o8.silu(G + h) * U - o8.silu(G - h) * U) / (2 * h)
    num_U = dH * (o8.silu(G) * (U + h) - o8.silu(G) * (U - h)) / (2 * h)
    # differences of second order: h^2 times a third derivative below 1, and
    # 2^-52 / h of cancellation
    assert np.allclose(dG, num_G, atol=2e-9, rtol=0) and np.allclose(dU, num_U, atol=2e-9, rtol=0)
