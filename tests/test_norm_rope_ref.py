"""The plain norms with positions that the GPU tests go by, against closed forms and differences (CPU only)."""
import numpy as np
import pytest

from tests import norm_rope_ref as ref


def setup(pairing, seed=0, d=8, pairs=3):
    g = np.random.default_rng(seed)
    x, dy, w = g.normal(size=(2, 5, 3, d)), g.normal(size=(2, 5, 3, d)), 1 + 0.3 * g.normal(size=d)
    positions = g.integers(-50, 50, (2, 2, 5))
    return x, dy, w, (1e-3, positions, g.uniform(0.01, 2, pairs), [0, 1, 1][:pairs], pairing)


def test_norm_alone():
    x, _, w, _ = setup("adjacent")
    y, _ = ref.forward(x, None, 0.0, np.zeros((1, 2, 5)), [], [], "adjacent")
    assert np.allclose((y * y).mean(-1), 1.0, rtol=1e-14)
    y2, _ = ref.forward(3.5 * x, w, 0.0, np.zeros((1, 2, 5)), [], [], "adjacent")
    assert np.allclose(y2, y * w, rtol=1e-13)


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_rotation_keeps_lengths(pairing):
    x, _, _, (eps, *tables) = setup(pairing)
    y, _ = ref.rotate(x, *tables)
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-13)
    assert np.allclose(ref.rotate(y, *tables, sign=-1.0)[0], x, rtol=0, atol=1e-13)


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_gradient_against_differences(pairing):
    x, dy, w, rest = setup(pairing, 1)
    dx, _, dw, _ = ref.backward(dy, x, w, *rest)
    loss = lambda x, w: (ref.forward(x, w, *rest)[0] * dy).sum()      # noqa: E731
    g, h = np.random.default_rng(2), 1e-5
    for _ in range(5):
        u, v = g.normal(size=x.shape), g.normal(size=w.shape)
        got = (loss(x + h * u, w) - loss(x - h * u, w)) / (2 * h), (loss(x, w + h * v) - loss(x, w - h * v)) / (2 * h)
        assert np.allclose(got, ((dx * u).sum(), (dw * v).sum()), rtol=1e-7)
