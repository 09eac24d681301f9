"""The oracle of layer norm, the gradients' norm and AdamW, against differences
and worked values (no GPU)."""
import numpy as np

from oracle import training_ops as Q


def _central(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_layer_norm_of_a_worked_row():
    x = np.array([[1.0, 2.0, 3.0, 6.0]])
    s, mean, rstd, y = Q.layer_norm(x, None, np.array([1.0, 1.0, 2.0, 1.0]), np.array([0.0, 1.0, 0.0, 0.0]), 0.5)
    assert mean[0] == 3.0 and np.isclose(rstd[0], 0.5)               # variance 3.5, eps 0.5
    assert np.allclose(y, [[-1.0, 0.5, 0.0, 1.5]])


def test_layer_norm_gradients_are_differences():
    rng = np.random.default_rng(3)
    x, r, w, b, dy, dsum = (rng.standard_normal(s) for s in ((3, 8), (3, 8), 8, 8, (3, 8), (3, 8)))
    eps = 0.01

    def loss(x, r, w, b):
        s, _, _, y = Q.layer_norm(x, r, w, b, eps)
        return (y * dy).sum() + (s * dsum).sum()
    s, mean, rstd, _ = Q.layer_norm(x, r, w, b, eps)
    ds, dw, db = Q.layer_norm_backward(dy, dsum, s, w, mean, rstd)
    # central differences: off by h^2 times third derivatives, and by 1e-16 / h
    for got, want in ((ds, _central(lambda v: loss(v, r, w, b), x)), (ds, _central(lambda v: loss(x, v, w, b), r)),
                      (dw, _central(lambda v: loss(x, r, v, b), w)), (db, _central(lambda v: loss(x, r, w, v), b))):
        assert np.allclose(got, want, rtol=1e-7, atol=1e-7)
