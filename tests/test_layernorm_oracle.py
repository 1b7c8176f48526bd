"""The fp64 oracle of the layer norm (oracle/layernorm.py) pinned by closed forms and differences.
Central differences with step 1e-5: error below 1e-6 (step^2 and rounding, losses of size 1e2)."""
import numpy as np

from oracle import layernorm


def test_two_values():
    """A row (m - c, m + c): mean m, variance c^2, y = -+ c / sqrt(c^2 + eps)."""
    y, mean, rstd = layernorm.forward(np.array([[4.0, 10.0]]), np.array([2.0, 3.0]), np.array([0.5, -0.5]), eps=0.0)
    assert np.allclose(y, [[-2.0 + 0.5, 3.0 - 0.5]], rtol=1e-14) and mean[0] == 7.0 and np.isclose(rstd[0], 1 / 3)


def test_constant_rows_and_one_column():
    y, mean, rstd = layernorm.forward(np.full((2, 5), 3.0), np.ones(5), np.arange(5.0), eps=1e-5)
    assert np.array_equal(y, np.tile(np.arange(5.0), (2, 1))) and np.allclose(rstd, 1e5 ** 0.5)
    y, _, _ = layernorm.forward(np.array([[8.0]]), np.array([2.0]), np.array([0.25]))
    assert y[0, 0] == 0.25


def test_gradients_against_differences():
    rng = np.random.default_rng(7)
    s, w, b = rng.standard_normal((3, 6)) * 2 + 1, rng.standard_normal(6), rng.standard_normal(6)
    dy, dres = rng.standard_normal((3, 6)), rng.standard_normal((3, 6))

    def loss(s, w, b):
        return float((layernorm.forward(s, w, b)[0] * dy).sum() + (s * dres).sum())
    _, mean, rstd = layernorm.forward(s, w, b)
    got = layernorm.grads(dy, s, w, mean, rstd, dres)
    for k, (v, name) in enumerate(((s, "ds"), (w, "dweight"), (b, "dbias"))):
        num = np.zeros_like(v)
        for at in np.ndindex(*v.shape):
            d = []
            for sign in (1.0, -1.0):
                args = [s, w, b]
                args[k] = v.copy()
                args[k][at] += sign * 1e-5
                d.append(loss(*args))
            num[at] = (d[0] - d[1]) / 2e-5
        assert np.abs(num - got[name]).max() < 1e-6, name
