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


def test_grad_norm():
    assert Q.grad_norm([np.array([3.0]), np.zeros((2, 0)), np.array([[4.0]])], 10) == (5.0, 1.0)
    assert Q.grad_norm([np.array([3.0, 4.0])], 1.0) == (5.0, 0.2)
    assert np.isnan(Q.grad_norm([np.array([np.inf])], 1.0)[1])


def test_mix_of_known_values():
    """MurmurHash3's finalizer: 0 stays 0, and it is a bijection with known images."""
    assert Q.mix(0) == 0 and Q.mix(1) == 0x514E28B7 and Q.mix(0xFFFFFFFF) == 0x81F16F39


def test_adamw_first_step_is_the_sign():
    """With zero moments the corrected m is g and the corrected v is g^2."""
    w, m, v = Q.adamw(np.array([1.0, -2.0]), np.array([0.3, -5.0]), np.zeros(2), np.zeros(2), 1, 0.1, (0.9, 0.99), 0.0, 0.5)
    assert np.allclose(w, [1 - 0.1 * (1 + 0.5), -2 - 0.1 * (-1 - 1.0)]) and np.allclose(m, [0.03, -0.5])
    assert np.allclose(v, [0.01 * 0.09, 0.25])


def test_random_bits_are_spread():
    """65536 elements: each bit is one in half of them, 6 standard deviations (768) either way; so is the exclusive or
    with the next element's, the next step's and the next tensor's."""
    a = Q.random_bits(5, 3, 2, 65536)
    for b in (np.zeros_like(a), np.roll(a, 1), np.roll(a, 128), Q.random_bits(5, 4, 2, 65536), Q.random_bits(5, 3, 3, 65536),
              Q.random_bits(6, 3, 2, 65536)):
        for bit in range(32):
            assert abs(int(((a ^ b) >> np.uint32(bit) & np.uint32(1)).sum()) - 32768) <= 768


def test_codes_are_right_on_average():
    """Every value between two codes, rounded 4096 times: a code step is at most 1/8 of the value above the subnormals,
    so 6 standard deviations of the mean are 6/2 * x / 8 / 64."""
    x = np.concatenate([[448.0], np.linspace(0.5, 300, 127)])
    r = Q.random_bits(1, 1, 1, 4096 * 128) >> np.uint32(16)
    mean = np.zeros(128)
    for k in range(4096):
        codes, scales, _ = Q.encode8(x, r[128 * k:128 * k + 128])
        mean += Q.decode8(codes, scales) / 4096
    assert np.all(np.abs(mean - x) <= 6 / 2 * x / 8 / 64)
    codes, scales, _ = Q.encode8(np.array([np.nan, -np.inf, 1.0, -1.0, 0.0]), r[:5])
    assert codes.tolist() == [127, 255, 126, 254, 0] and scales[0] == 1 / 448
    assert np.isnan(Q.decode8(codes, scales)[:2]).all()


def test_8bit_second_moments_follow_the_gradients():
    """Normal gradients for several times 1 / (1 - beta2) steps: v stays with the exact average, larger by the rounding's
    variance.  The rounding adds at most s^2 f with s <= 1/8 of r the distance of two codes and f = (1 - beta2)
    |g^2 - v| / (2 r) / s the part of the way that a step goes, at most (1 - beta2) |g^2 - v| / 16 a step, which decays
    by 1 - beta2: at most 1/16 of E|g^2 - v|, which is about v: 0.07 with the spread that v itself has."""
    rng = np.random.default_rng(0)
    scale = np.exp(rng.uniform(-2, 0, 1024))
    for beta2, steps in ((0.95, 300), (0.999, 3000)):
        codes, scales, exact = np.zeros(1024, np.uint8), np.zeros(8), np.zeros(1024)
        for t in range(1, steps + 1):
            g = scale * rng.standard_normal(1024)
            exact = beta2 * exact + (1 - beta2) * g * g
            v = beta2 * Q.decode8(codes, scales) ** 2 + (1 - beta2) * g * g
            codes, scales, _ = Q.encode8(np.sqrt(v), Q.random_bits(9, t, 0, 1024) >> np.uint32(16))
        ratio = (Q.decode8(codes, scales) ** 2).sum() / exact.sum()
        assert 0.95 <= ratio <= 1.1, (beta2, ratio)
