"""8-bit moments of blocks whose elements differ by many orders of magnitude (marked gpu)."""
import numpy as np
import pytest
import torch

from oracle import training_ops as Q
from routing_dispatch_grouped_router_amd import binding as B
from routing_dispatch_grouped_router_amd.workloads import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


@pytest.mark.parametrize("n", [128, 1000, 4097])
@pytest.mark.parametrize("w", [torch.float32, torch.bfloat16])
def test_codes_of_small_roots(n, w):
    """The first step from zero: roots over eighteen orders of magnitude; 0 stays 0, nothing else becomes it.  Past
    that the codes are the oracle's, but for places that 12 roundings of a value and of its block's largest (16 places
    a relative error at most) can move over a border."""
    print(f"[8-bit range] n={n} {w}", flush=True)
    rng = np.random.default_rng(n)
    g = (rng.standard_normal(n) * 10 ** rng.uniform(-17, 1, n)).astype(np.float32)
    g[rng.random(n) < 0.2] = 0
    op = B.AdamW([torch.zeros(n, dtype=w, device=DEV)], [torch.from_numpy(g).to(DEV)], lr=0.0, betas=(0.9, 0.95),
                 weight_decay=0.0, states="8bit", seed=3)
    op()
    torch.cuda.synchronize()
    got = op.r[0].cpu().numpy().astype(int)
    assert np.array_equal(got > 0, g != 0)
    bits = Q.random_bits(3, 1, 0, n)
    want, _, place = Q.encode8(np.sqrt(0.05) * np.abs(g.astype(np.float64)), bits >> np.uint32(16), root=True)
    off = got != want.astype(int)
    near = np.abs(place - np.round(place)) <= 16 * 24 * U + 2.0 ** -20
    assert np.all(~off | (near & (np.abs(got - want.astype(int)) <= 1))), f"{off.sum()} codes off"


@pytest.mark.parametrize("spread", [1e-4, 1e-5, 1e-6, 1e-7])
def test_steps_of_small_elements_stay_bounded(spread):
    """Half of each block's gradients are `spread` times the others, 300 steps with betas 0.9 and 0.95.  Moments in full
    precision make steps of 1.17 lr at most: |m| <= (1 - b1) sqrt(sum of (b1^2 / b2)^i) sqrt(v / (1 - b2)), 0.447 sqrt(6.79)
    (at the first steps 1).  A rounding takes m / sqrt(v) to twice itself and the ratio of the block's largest values at
    most (m a code up, the root one down but not below 1): 3.5."""
    rng, n, lr = np.random.default_rng(2), 1024, 2.0 ** -10
    scale = np.where(np.arange(n) % 2 == 0, 1.0, spread)
    w, g = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    op = B.AdamW([w], [g], lr=lr, betas=(0.9, 0.95), weight_decay=0.0, states="8bit", seed=9)
    worst, before = 0.0, as_f64(w)
    for _ in range(300):
        g.copy_(torch.from_numpy((scale * rng.standard_normal(n)).astype(np.float32)))
        op()
        after = as_f64(w)
        worst, before = max(worst, np.abs(after - before).max() / lr), after
    assert worst <= 3.5, worst


def test_scales_and_codes_are_the_formulas():
    """With beta1 0 the moment is the gradient.  Its scale is amax (1 / 448) and its place |x| (448 (1 / amax)), every
    reciprocal and product a float32."""
    blocks = 4096
    rng = np.random.default_rng(5)
    g = (rng.standard_normal((blocks, 128)) * 10 ** rng.uniform(-6, 6, (blocks, 1))).astype(np.float32)
    op = B.AdamW([torch.zeros(blocks * 128, device=DEV)], [torch.from_numpy(g.reshape(-1)).to(DEV)], lr=0.0, betas=(0.0, 0.95),
                 weight_decay=0.0, states="8bit", seed=21)
    op()
    torch.cuda.synchronize()
    amax = np.abs(g).max(axis=1)
    assert np.array_equal(op.m_scale[0].cpu().numpy(), amax * (np.float32(1) / np.float32(448)))
    a = np.minimum(np.abs(g) * (np.float32(448) * (np.float32(1) / amax))[:, None], np.float32(448)).reshape(-1).astype(np.float64)
    c = np.minimum(np.searchsorted(Q.E4M3, a, side="right") - 1, 125)
    r16 = (Q.random_bits(21, 1, 0, a.size) & np.uint32(0xFFFF)).astype(np.float64)
    place = c + (a - Q.E4M3[c]) / (Q.E4M3[c + 1] - Q.E4M3[c])
    codes = np.minimum(np.floor(place + (r16 + 0.5) / 65536), 126).astype(int) + np.where(g.reshape(-1) < 0, 128, 0)
    # float32 has 20 bits below a code's last: a denormal or rounded sum of place and random bits is 2^-20 off at most
    sure = np.abs((place + (r16 + 0.5) / 65536) - np.round(place + (r16 + 0.5) / 65536)) > 2.0 ** -20
    assert sure.mean() > 0.99 and np.array_equal(op.m[0].cpu().numpy().astype(int)[sure], codes[sure])
