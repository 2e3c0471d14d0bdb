"""Pins of the oracle's norm, rotation and quantisation (CPU): identities that do not use its own code."""
import numpy as np
import pytest

from oracle import prep


def _angles(n, d, seed):
    a = np.random.default_rng(seed).uniform(-100, 100, (n, d // 2))
    return a, np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_multiplication_by_a_unit_complex_number(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 16))
    a, c, s = _angles(5, 16, 2)
    y = prep.rotate(x, c, s, interleaved)
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 8), slice(8, 16))
    z = (x[:, first] + 1j * x[:, second]) * np.exp(1j * a)
    np.testing.assert_allclose(y[:, first] + 1j * y[:, second], z, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_products_depend_on_the_distance_alone(interleaved):
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((2, 8))
    f = rng.uniform(0.1, 1, 4)
    dot = lambda p, r: prep.rotate(q, np.cos(p * f), np.sin(p * f), interleaved) @ prep.rotate(  # noqa: E731
        k, np.cos(r * f), np.sin(r * f), interleaved)
    assert abs(dot(7, 3) - dot(104, 100)) < 1e-12
    assert abs(dot(7, 3) - dot(7, 4)) > 1e-3


def test_norms():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((3, 32)) * 7 + 2
    y = prep.rms_norm(x, np.ones(32), 0.0)
    np.testing.assert_allclose((y * y).mean(-1), 1, rtol=1e-12)
    z = prep.layer_norm(x, np.ones(32), np.zeros(32), 0.0)
    np.testing.assert_allclose(z.mean(-1), 0, atol=1e-12)
    np.testing.assert_allclose(z.std(-1), 1, rtol=1e-12)
    np.testing.assert_allclose(prep.layer_norm(x, 2 * np.ones(32), 3 * np.ones(32), 0.0), 2 * z + 3, rtol=1e-12)


def test_quantise_reaches_the_top_code_and_keeps_zero():
    z = np.array([[1.0, -4.0, 2.0], [0.0, 0.0, 0.0]])
    v, s = prep.quantise(z, 448.0)
    np.testing.assert_allclose(v * s[:, None], z)
    assert v[0].min() == -448 and s[1] == 1
