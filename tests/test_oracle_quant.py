"""Pins of the fp64 reference of quantised pages (no GPU)."""
import numpy as np
import torch

from oracle import quant


def test_values_are_the_type_s():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(quant.VALUES, want)


def test_exponent_by_hand():
    assert quant.exponent(448.0) == 0 and quant.exponent(448.0001) == 1
    assert quant.exponent(224.0) == -1 and quant.exponent(1.0) == -8
    assert quant.exponent(1.75) == -8 and quant.exponent(1.7501) == -7
    assert quant.exponent(0.0) == -64 and quant.exponent(1e300) == 63


def test_rounding_is_to_nearest_even_and_by_at_most_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * 2.0 ** rng.integers(-30, 30, (200, 1))
    codes, scale = quant.quantise(x)
    y = quant.value(codes, scale)
    e = scale.astype(int) - 127
    assert [quant.exponent(a) for a in np.abs(x).max(-1)] == e.tolist()
    step = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * 2.0 ** e[:, None])
    assert np.all(np.abs(y - x) <= step)
    # against the type's own conversion
    t = torch.from_numpy(x * 2.0 ** -e[:, None]).float().to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(codes, t.view(torch.uint8).numpy())


def test_special_values():
    codes, scale = quant.quantise(np.array([[np.inf, -np.nan, -0.0, 1.0], [0, 0, 0, 0.0],
                                            [1e30, -1e30, 1.0, 0.0]]))
    assert (codes[0, :2] & 127 == 127).all() and codes[0, 2] == 128
    assert quant.value(codes, scale)[0, 3] == 1.0
    assert scale[1] == 63 and not codes[1].any()
    assert codes[2].tolist() == [126, 254, 0, 0] and scale[2] == 190


def test_norm_by_hand():
    x = np.array([[3.0, 4.0]])
    np.testing.assert_allclose(quant.norm(x, np.array([1.0, 2.0]), 0.0),
                               [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    assert quant.norm(x, None, 1.0) is not None
