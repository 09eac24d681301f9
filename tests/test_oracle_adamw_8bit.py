"""8-bit moments of blocks whose elements differ by many orders of magnitude, in the oracle (no GPU).

A root's smallest code is its block's largest value / 229376, a moment's is too, and each is rounded at random.  Were
a positive root left without a code while its element's m has one, the next step would divide m by nearly nothing."""
import numpy as np
import pytest

from oracle import training_ops as Q

EPS = 1e-8


def largest_step(betas, steps):
    """The largest |m c1 / sqrt(v c2)| that `steps` gradients can make of moments in full precision: by Cauchy and
    Schwarz |m| <= (1 - b1) sqrt(sum of (b1^2 / b2)^i) sqrt(v / (1 - b2)) after t steps, i < t."""
    b1, b2 = betas
    t = np.arange(1, steps + 1)
    q = b1 * b1 / b2
    ratio = (1 - b1) / np.sqrt(1 - b2) * np.sqrt((1 - q ** t) / (1 - q))
    return np.max(ratio * np.sqrt(1 - b2 ** t) / (1 - b1 ** t))


# a rounding leaves m at most a code above its place and a root at most one below, never below 1: in units of the
# smallest codes m' <= m + 1 and r' >= max(1, r / 2), so that one rounding takes m / r to 2 m / r plus the ratio of the
# two blocks' largest values at most, three times the largest step
ROUNDED = 3


@pytest.mark.parametrize("betas", [(0.9, 0.95), (0.9, 0.99), (0.9, 0.999)])
@pytest.mark.parametrize("spread", [1e-4, 1e-5, 1e-6, 1e-7])
@pytest.mark.parametrize("size", [1.0, 1e-2])
def test_steps_of_small_elements_stay_bounded(betas, spread, size):
    """Half of each block's gradients are `spread` times the others; 500 steps."""
    rng, n, steps = np.random.default_rng(1), 1024, 500
    scale = size * np.where(np.arange(n) % 2 == 0, 1.0, spread)
    m8 = r8 = np.zeros(n, np.uint8)
    ms = rs = np.zeros(n // Q.BLOCK)
    worst = 0.0
    for t in range(1, steps + 1):
        step, m, v = Q.adamw(np.zeros(n), scale * rng.standard_normal(n), Q.decode8(m8, ms), Q.decode8(r8, rs) ** 2, t, 1.0,
                             betas, EPS, 0.0)
        worst = max(worst, np.abs(step).max())
        bits = Q.random_bits(9, t, 0, n)
        m8, ms, _ = Q.encode8(m, bits & np.uint32(0xFFFF))
        r8, rs, _ = Q.encode8(np.sqrt(v), bits >> np.uint32(16), root=True)
    assert worst <= ROUNDED * largest_step(betas, steps)


def test_codes_of_small_roots():
    """A positive root has a code of 1 at least, a zero none; moments and larger roots are rounded as they were."""
    x = np.array([448.0, 1 / 512, 1e-9, 0.0, 1e-300, 0.3 / 512, np.inf, np.nan] + [0.0] * 120 + [0.0, 2.0 ** -101] + [0.0] * 126)
    r16 = np.zeros(256, np.uint32)
    codes, scales, place = Q.encode8(x, r16, root=True)
    assert codes[:8].tolist() == [126, 1, 1, 0, 1, 1, 127, 127] and scales.tolist() == [1.0, 0.0]
    assert not codes[8:].any()                         # a block below 2^-100 is zero
    plain, again, same = Q.encode8(x, r16)
    assert plain[:8].tolist() == [126, 1, 0, 0, 0, 0, 127, 127]
    assert np.array_equal(again, scales) and np.array_equal(same, place)
