"""Infinite, NaN and very large operands of moe_router_backward (marked gpu):
the gradients they reach are what the sums of products give (an infinity of
its sign, or NaN where it meets a zero or the opposite infinity), the others
stay as they are.

Tolerances of the finite values as in the router's other tests: products of n
terms in float32, each in up to six partial products, 6 n + 16 half-steps of
the sum of magnitudes, dx rounded once to its type."""
import numpy as np
import pytest
import torch

from routing_dispatch_grouped_router_amd import binding as B
from routing_dispatch_grouped_router_amd.workloads import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
INF = float("inf")


def _draws(rng):
    return lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))


def _products(a, b):
    """a b of float64 matrices, infinities and NaN by the rules of a sum of products."""
    with np.errstate(invalid="ignore"):
        return np.stack([(a[:, :, None] * b[None, :, j:j + 1]).sum(1)[:, 0] for j in range(b.shape[1])], 1)


def _same(name, got, ref, tol):
    got = as_f64(got)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{name}: NaN in {np.argwhere(np.isnan(got) != np.isnan(ref))[:5]}"
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), name
    bad = ~(np.abs(got[fin] - ref[fin]) <= tol[fin])
    assert not bad.any(), f"{name}: {bad.sum()} values off"


def _check(dl, x, w, a, act):
    T, E, d = dl.shape[0], dl.shape[1], x.shape[1]
    op = B.RouterBackward(B.problem(T, d, E, 1, 64, act), DEV)
    op.ws.fill_(255)
    g = op(dl.to(DEV), x.to(DEV), w.to(DEV), dx_in=None if a is None else a.to(DEV))
    dl64, x64, w64 = (as_f64(t) for t in (dl, x, w))
    ref, mag = _products(dl64, w64.T), _products(np.abs(dl64), np.abs(w64.T))
    if a is not None:
        ref, mag = ref + as_f64(a), mag + np.abs(as_f64(a))
    half = 2.0 ** -24 if act == "f32" else 2.0 ** -8
    with np.errstate(invalid="ignore"):
        _same("dx", g["dx"], ref, half * np.abs(ref) + (6 * E + 16) * U * mag)
        ref, mag = _products(x64.T, dl64), _products(np.abs(x64.T), np.abs(dl64))
        # up to 512 ranges of T / 512 tokens (rounded up by less than 160), added after
        _same("dw_router", g["dw_router"], ref, (6 * (T / 512 + 160) + 512 + 64) * U * mag)
    if a is not None:                                         # in place
        want = {k: v.clone() for k, v in g.items()}
        op.dx = a.to(DEV)
        g = op(dl.to(DEV), x.to(DEV), w.to(DEV), dx_in=op.dx)
        assert all(torch.allclose(g[k], want[k], rtol=0, atol=0, equal_nan=True) for k in want)


# the resident kernel (bf16, up to 64 experts: one and two 32's), the general one, one token range and several
@pytest.mark.parametrize("T, d, E, act", [(70, 128, 8, "bf16"), (300, 320, 40, "bf16"), (300, 64, 100, "bf16"),
                                          (70, 128, 8, "f32"), (300, 64, 33, "f32"), (1, 64, 1, "bf16"), (1, 64, 1, "f32")])
@pytest.mark.parametrize("add", [False, True])
def test_infinities_and_nan(T, d, E, act, add):
    print(f"[nonfinite router gradients] T={T} d={d} E={E} {act} add={add}", flush=True)
    rng = np.random.default_rng(T + d + E)
    dt = B.storage_dtype(act)
    draw = _draws(rng)
    base = [draw(T, E), draw(T, d).to(dt), draw(d, E).to(dt)]
    base[0][T // 2] = 0                                       # a token without a gradient
    base[0][T // 3, E // 2] = 1.0                             # one bfloat16 term, its remainders zero
    a = draw(T, d).to(dt) if add else None
    for which in range(3):
        for value in (INF, -INF, float("nan")):
            for spot in (0, 1):
                ops = [t.clone() for t in base]
                t = ops[which]
                t[(0 if spot == 0 else t.shape[0] // 3), (0 if spot == 0 else t.shape[1] // 2)] = value
                _check(*ops, a, act)
    ops = [t.clone() for t in base]                           # an infinite x at a token whose gradients are all zero
    ops[1][T // 2, d - 1] = INF
    _check(*ops, a, act)
    ops = [t.clone() for t in base]                           # infinities that meet
    ops[0][0, 0], ops[0][T - 1, 0] = INF, -INF
    _check(*ops, a, act)
    if add:
        a[0, 1], a[T - 1, d - 1] = INF, -INF
        _check(*base, a, act)


@pytest.mark.parametrize("T, d, E, act", [(70, 128, 8, "bf16"), (130, 64, 72, "bf16"), (70, 128, 9, "f32")])
def test_values_above_bfloat16s_largest(T, d, E, act):
    rng = np.random.default_rng(E)
    dt = B.storage_dtype(act)
    draw = _draws(rng)
    top = float(np.finfo(np.float32).max)
    for value in (top, -top, float(np.float32(3.3953e38))):
        dl, x, w = draw(T, E), draw(T, d).to(dt), draw(d, E).to(dt)
        x, w = x * 2.0 ** -10, w * 2.0 ** -10
        dl[3, E - 1] = value
        _check(dl, x, w, None, act)
        if act == "f32":
            dl, w = draw(T, E) * 2.0 ** -10, draw(d, E)
            x = draw(T, d)
            x[5, 0] = value
            _check(dl, x, w, None, act)
            x, w = draw(T, d), draw(d, E)
            w[5, 0] = value
            _check(dl, x, w, None, act)


# several tiles of tokens a workgroup, through the caches and past them
@pytest.mark.parametrize("T, d, E", [(70001, 64, 20), (262300, 64, 40)])
def test_infinities_among_many_tokens(T, d, E):
    print(f"[nonfinite router gradients] T={T} d={d} E={E}", flush=True)
    g = torch.Generator().manual_seed(T)
    dl = torch.randn(T, E, generator=g).to(DEV)
    x, w, a = (torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV) for s in ((T, d), (d, E), (T, d)))
    op = B.RouterBackward(B.problem(T, d, E, 1, 64, "bf16"), DEV)
    good = {k: v.clone() for k, v in op(dl, x, w, dx_in=a).items()}
    rows = torch.tensor([3, 70, 40000, T - 70, T - 1], device=DEV)
    dl[rows, 1] = INF
    op.dx = a.clone()
    got = op(dl, x, w, dx_in=op.dx)
    dx, dw = good["dx"].clone(), good["dw_router"].clone()
    dx[rows] = (INF * w[:, 1]).expand(len(rows), d)           # (no zero among w's or x's values here)
    lo, hi = x[rows].float().amin(0), x[rows].float().amax(0)
    dw[:, 1] = torch.where(lo > 0, INF, torch.where(hi < 0, -INF, float("nan")))
    assert w[:, 1].all() and x[rows].all()
    assert torch.allclose(got["dx"], dx, rtol=0, atol=0, equal_nan=True)
    assert torch.allclose(got["dw_router"], dw, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_infinite_gradient_from_another_loss(act):
    """moe_backward_aux, whose dx adds gathered rows to the product."""
    T, d, E, k, H = 200, 128, 12, 3, 128
    rng = np.random.default_rng(8)
    dt, p = B.storage_dtype(act), B.problem(T, d, E, k, H, act)
    draw = lambda *s, scale=1.0: torch.from_numpy((scale * rng.standard_normal(s)).astype(np.float32)).to(dt).to(DEV)
    x, wr, dy = draw(T, d), draw(d, E, scale=0.05), draw(T, d)
    ws = [draw(E, d, H, scale=0.05), draw(E, d, H, scale=0.05), draw(E, H, d, scale=0.05)]
    packed, packed_bwd = B.pack_weights(p, *ws), B.pack_weights_backward(p, *ws)
    fwd, bwd = B.Forward(p, DEV), B.Backward(p, DEV, aux=True)
    fwd(x, packed=packed, w_router=wr)
    aux = torch.zeros((T, E), device=DEV)

    def run():
        g = bwd(fwd, dy, packed, packed_bwd, x=x, w_router=wr, dlogits_aux=aux)
        return {n: g[n].clone() for n in ("dx", "dw_router")}
    good = run()
    rows = torch.tensor([0, 65, T - 1], device=DEV)
    aux[rows, 2] = -INF
    got = run()
    dx, dw = good["dx"].clone(), good["dw_router"].clone()
    dx[rows] = (-INF * wr[:, 2]).expand(3, d)
    lo, hi = x[rows].float().amin(0), x[rows].float().amax(0)
    dw[:, 2] = torch.where(lo > 0, -INF, torch.where(hi < 0, INF, float("nan")))
    assert torch.allclose(got["dx"], dx, rtol=0, atol=0, equal_nan=True)
    assert torch.allclose(got["dw_router"], dw, rtol=0, atol=0, equal_nan=True)
