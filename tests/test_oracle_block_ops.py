"""Pins of the oracle of the operators around the block (oracle/block_ops.py):
its gradients against differences of its forwards, its MXFP4 format against
the definition's worked values.  CPU only."""
import numpy as np
import pytest

from oracle import block_ops as Q

RNG = np.random.default_rng(7)


def _numeric(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("residual", [False, True])
def test_norm_gradient_is_the_difference_quotient(residual):
    x, w, dy = RNG.standard_normal((3, 8)), RNG.standard_normal(8), RNG.standard_normal((3, 8))
    r = RNG.standard_normal((3, 8)) if residual else None
    eps = 1e-3
    s, rstd, _ = Q.rmsnorm(x, r, w, eps)
    dsum = RNG.standard_normal((3, 8))
    ds, dw = Q.rmsnorm_backward(dy, dsum, s, w, rstd=rstd)

    def loss(xx, ww=w):
        ss, _, y = Q.rmsnorm(xx, r, ww, eps)
        return (y * dy).sum() + (ss * dsum).sum()
    np.testing.assert_allclose(ds, _numeric(loss, x), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dw, _numeric(lambda ww: loss(x, ww), w), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("mask", [None, [1, 0, 1, 1, 0]])
def test_balance_gradient_is_the_difference_quotient(mask):
    logits = RNG.standard_normal((5, 6))
    idx = np.argsort(-logits, axis=1)[:, :2]
    m = None if mask is None else np.array(mask, np.uint8)
    _, counts, n = Q.balance_loss(logits, idx, m)
    g = (0.7, 0.3)
    dl = Q.balance_loss_backward(logits, counts, 2, g, m)

    def loss(l):   # the choices stay as they are
        out, _, _ = Q.balance_loss(l, idx, m)
        return g[0] * out[0] + g[1] * out[1]
    np.testing.assert_allclose(dl, _numeric(loss, logits), rtol=1e-6, atol=1e-8)
    assert n == (5 if mask is None else 3) and counts.sum() == 2 * n


def test_balance_of_even_routing_is_one():
    logits = np.zeros((8, 4))
    idx = (np.arange(8)[:, None] + np.arange(2)) % 4
    loss, counts, _ = Q.balance_loss(logits, idx)
    assert loss[0] == pytest.approx(1.0) and loss[1] == pytest.approx(np.log(4) ** 2)
    assert counts.tolist() == [4, 4, 4, 4]


def test_balance_without_live_tokens_or_finite_logits():
    logits = np.full((2, 3), np.nan)
    loss, counts, n = Q.balance_loss(logits, np.zeros((2, 1), int), np.zeros(2))
    assert loss.tolist() == [0, 0] and counts.sum() == 0 and n == 0
    p, lse = Q._softmax(np.array([[-np.inf, -np.inf], [0.0, -np.inf]]))
    assert p.tolist() == [[0, 0], [1, 0]] and lse.tolist() == [0, 0]


def test_mxfp4_worked_block():
    v = np.zeros(32)
    # amax 5 -> shared exponent 2 - 2 = 0: the elements themselves are rounded
    v[:12] = [5.0, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -4.5, 0.26, -0.0, 4.9, 5.1]
    c, s = Q.mxfp4_quantize(v)
    assert s.tolist() == [127]
    got = Q.mxfp4_values(c, s)[:12]
    assert got.tolist() == [4.0, -0.0, 1.0, 1.0, 2.0, 2.0, 4.0, -4.0, 0.5, -0.0, 4.0, 6.0]
    assert np.signbit(got[[1, 9]]).all()
    # amax 7 keeps exponent 0 and saturates to 6; zero blocks take the smallest scale
    c, s = Q.mxfp4_quantize(np.array([7.0] + [0.0] * 31 + [0.0] * 32))
    assert s.tolist() == [127, 0] and Q.mxfp4_values(c, s)[0] == 6.0
    assert Q.unpack_codes(np.array([0x7F, 0x10], np.uint8)).tolist() == [15, 7, 0, 1]


def test_mxfp4_scaled_by_powers_of_two():
    v = RNG.standard_normal((4, 64))
    c, s = Q.mxfp4_quantize(v)
    for e in (-40, 17):
        c2, s2 = Q.mxfp4_quantize(np.ldexp(v, e))
        assert np.array_equal(c, c2) and np.array_equal(s.astype(int) + e, s2.astype(int))
    assert np.max(np.abs(Q.mxfp4_values(c, s) - v) / np.abs(v).reshape(4, 2, 32).max(2).repeat(32, 1)) <= 0.25
