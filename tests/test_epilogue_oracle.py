"""The epilogue oracle against closed forms, and the slope bound that its tolerance uses."""
import math

import numpy as np
import pytest

from oracle import epilogue as oepi


def test_activations_at_known_points():
    assert oepi.activation(np.array([-2.0, 0.0, 3.0]), "relu").tolist() == [0.0, 0.0, 3.0]
    assert oepi.activation(np.array([0.0]), "silu")[0] == 0.0
    assert oepi.activation(np.array([math.log(3)]), "silu")[0] == pytest.approx(0.75 * math.log(3), rel=1e-15)
    # Phi(1) = 0.8413447460685429
    assert oepi.activation(np.array([1.0]), "gelu")[0] == pytest.approx(0.8413447460685429, rel=1e-14)
    z = math.sqrt(2 / math.pi) * 1.044715
    want = 0.5 * (1 + (math.exp(z) - math.exp(-z)) / (math.exp(z) + math.exp(-z)))
    assert oepi.activation(np.array([1.0]), "gelu_tanh")[0] == pytest.approx(want, rel=1e-14)
    # Phi(z) + Phi(-z) = 1, so gelu(z) - gelu(-z) = z; the same holds for tanh and the sigmoid
    g = np.linspace(-5, 5, 41)
    for name in ("gelu", "gelu_tanh", "silu"):
        np.testing.assert_allclose(oepi.activation(g, name) - oepi.activation(-g, name), g, atol=1e-13)


def test_nan_passes_every_activation():
    for name in oepi.ACTIVATIONS:
        assert np.isnan(oepi.activation(np.array([np.nan]), name)[0])


@pytest.mark.parametrize("name", oepi.ACTIVATIONS)
def test_slope_bound(name):
    z = np.linspace(-12, 12, 200001)
    a = oepi.activation(z, name)
    assert np.max(np.abs(np.diff(a) / np.diff(z))) <= oepi.MAX_SLOPE


def test_apply_is_the_formula_by_hand():
    v = np.array([[1.0, -2.0]])
    y, tol = oepi.apply(v, bias=np.array([1.0, 1.0]), act="relu", residual=np.array([[0.5, 0.25]]))
    assert y.tolist() == [[2.5, 0.25]]
    assert (tol > 0).all() and (tol < 0.02).all()
