"""The oracle of the normed rotary positions: its gradients against central
differences of its forward, and closed forms."""
import numpy as np
import pytest

from oracle import norm as O


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_against_differences(interleaved):
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal((2, 2, 3, 6)), rng.standard_normal((2, 2, 3, 6))
    w = 1.0 + 0.3 * rng.standard_normal(6)
    pos, freqs = np.array([[0, 5, -9]] * 2), np.array([1.0, 0.03])
    args = (pos, freqs, interleaved, 1.25, 1e-3)
    dx, dw = O.backward(g, x, w, *args)
    loss = lambda x, w: (O.forward(x, w, *args) * g).sum()
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(6):
        e = np.zeros_like(w)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_closed_forms():
    x = np.full((1, 1, 1, 4), 3.0)
    none = np.zeros((1, 1))
    assert np.allclose(O.forward(x, None, none, [], eps=0.0), 1.0)
    assert np.allclose(O.forward(0 * x, None, none, [], eps=1e-6), 0.0)
    # along x nothing changes: the gradient of a head's direction has no part along it
    dx, _ = O.backward(x, x, None, none, [], eps=0.0)
    assert np.allclose(dx, 0.0)
