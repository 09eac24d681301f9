"""The router's losses and dense gradients (moe_balance_loss and its backward,
moe_router_backward) against their float64 oracle (marked gpu).

Tolerances in half-steps u = 2^-24 of the sum of magnitudes of what is added:
the loss's sums run over at most 160 tokens a lane (T = 40000, E = 8), 6 tree
steps, 16 waves, 256 / 8 workgroup sums in 16 chunks and E terms in trees: 400.  A softmax value is off by the rounding of its
exponent's argument, |l - max| u, and some ulps: 64 + 2 range.  Matrix products
of K terms in float32, each in up to six partial products: 6 K + 16."""
import numpy as np
import pytest
import torch

from oracle import block_ops as Q
from routing_dispatch_grouped_router_amd import binding as B
from routing_dispatch_grouped_router_amd.workloads import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


def _close(name, got, ref, tol):
    got = as_f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} values off, worst {np.max(np.abs(got - ref) - tol):.3e}"


def _balance_problem(T, E, k):
    return B.problem(T, 64, E, k, 64, "f32")


def _check_balance(logits, idx, mask, k, dloss=(0.3, 0.05)):
    T, E = logits.shape
    op = B.BalanceLoss(_balance_problem(T, E, k), DEV)
    op.ws.fill_(255)
    op.dlogits.fill_(float("nan"))
    l, i = torch.from_numpy(logits).to(DEV), torch.from_numpy(idx).to(DEV)
    m = None if mask is None else torch.from_numpy(mask).to(DEV)
    g = torch.tensor(dloss, dtype=torch.float32, device=DEV)
    op(l, i, mask=m)
    dl = op.backward(l, g, mask=m)
    torch.cuda.synchronize()
    l64, g64 = logits.astype(np.float64), as_f64(g)
    loss, counts, n = Q.balance_loss(l64, idx, mask)
    assert np.array_equal(op.counts.cpu().numpy(), counts) and int(op.live.item()) == n
    _close("loss", op.loss, loss, 400 * U * np.abs(loss))
    ref = Q.balance_loss_backward(l64, counts, k, g64, mask)
    live = np.ones(T, bool) if mask is None else mask != 0
    tol = np.zeros((T, E))
    if n:
        ll = l64[live]
        p, lse = Q._softmax(ll)
        f = counts / (n * k)
        fin = np.where(np.isfinite(ll), ll, np.nan)
        span = np.nan_to_num(np.nanmax(fin, 1, initial=-np.inf, where=~np.isnan(fin))[:, None] - fin, nan=0.0,
                             posinf=0.0, neginf=0.0)
        mag = p / n * (abs(g64[0]) * E * (f + (p * f).sum(1, keepdims=True)) + 2 * abs(g64[1]) * np.abs(lse)[:, None])
        # float32 probabilities below 2^-126 lose bits: an absolute 2^-126 on p
        tol[live] = (64 + 2 * np.minimum(span, 100)) * U * mag + 2.0 ** -126 / n * (E + 2 * np.abs(lse)[:, None])
    _close("dlogits", dl, ref, tol)
    assert not as_f64(dl)[~live].any()
    want = dl.clone()
    op.dlogits = l                                           # in place
    assert torch.equal(op.backward(l, g, mask=m), want)


# the lanes-per-token variants (E 1 .. 1024), token counts of one workgroup and of many
@pytest.mark.parametrize("T, E, k", [(1, 1, 1), (1, 4, 4), (5, 3, 2), (300, 8, 2), (1000, 12, 3), (777, 20, 4),
                                     (2049, 64, 8), (700, 128, 4), (513, 200, 6), (300, 260, 16), (40, 1024, 16),
                                     (40000, 8, 2), (70, 301, 3), (200, 512, 4), (90, 513, 2), (150, 700, 4)])
@pytest.mark.parametrize("padded", ["no", "some", "all"])
def test_balance(T, E, k, padded):
    print(f"[balance] T={T} E={E} k={k} padded={padded}", flush=True)
    rng = np.random.default_rng(T + E)
    logits = (2 * rng.standard_normal((T, E)) - np.linspace(0, 3, E)).astype(np.float32)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    mask = None
    if padded != "no":
        mask = (rng.random(T) < 0.7).astype(np.uint8) if padded == "some" else np.zeros(T, np.uint8)
        mask[mask != 0] = rng.integers(1, 256, int((mask != 0).sum()))   # any nonzero byte is live
        logits[mask == 0] = rng.choice([np.nan, np.inf, -np.inf], (int((mask == 0).sum()), 1))
        idx[mask == 0] = rng.integers(-2 ** 31, 2 ** 31 - 1, (int((mask == 0).sum()), k))
    _check_balance(logits, idx, mask, k)


def test_balance_of_excluded_experts_extremes_and_unused_choices():
    rng = np.random.default_rng(3)
    T, E, k = 200, 12, 3
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[:, 4] = -np.inf                                   # an excluded expert
    logits[5] = -np.inf                                      # a row without any
    logits[6] = np.float32(-1e18)                            # large, all equal (lse^2 still finite)
    logits[7, 2] = np.float32(3e18)
    logits[8, :6] = np.finfo(np.float32).min                 # the type's lowest value
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    idx[9] = -1
    idx[10, 1] = E
    idx[11] = 0                                              # the same expert thrice
    _check_balance(logits, idx, None, k, dloss=(0.3, 0.0))
    logits[6:8] = 0
    _check_balance(logits, idx, None, k)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T, d, E", [(1, 64, 1), (3, 128, 5), (64, 64, 8), (65, 192, 16), (200, 320, 17), (333, 256, 33),
                                     (1000, 576, 64), (2100, 256, 100), (130, 64, 520), (4100, 128, 8)])
@pytest.mark.parametrize("add", [False, True])
def test_router_backward(T, d, E, act, add):
    print(f"[router backward] T={T} d={d} E={E} {act} add={add}", flush=True)
    rng = np.random.default_rng(T + d + E)
    dt = B.storage_dtype(act)
    dl = torch.from_numpy((rng.standard_normal((T, E)) * 10.0 ** rng.integers(-6, 1, (T, E))).astype(np.float32))
    x, w, a = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dt) for s in ((T, d), (d, E), (T, d)))
    op = B.RouterBackward(B.problem(T, d, E, 1, 64, act), DEV)
    op.ws.fill_(255)
    dev = [t.to(DEV) for t in (dl, x, w)]
    add_dev = a.to(DEV) if add else None
    g = op(*dev, dx_in=add_dev)
    first = {k: v.clone() for k, v in g.items()}
    op(*dev, dx_in=add_dev)
    torch.cuda.synchronize()
    assert all(torch.equal(first[k], g[k]) for k in g)
    dl64, x64, w64, a64 = (as_f64(t) for t in (dl, x, w, a))
    ref = dl64 @ w64.T + (a64 if add else 0)
    mag = np.abs(dl64) @ np.abs(w64).T + (np.abs(a64) if add else 0)
    half = 2.0 ** -24 if act == "f32" else 2.0 ** -8
    _close("dx", g["dx"], ref, half * np.abs(ref) + (6 * E + 16) * U * mag)
    # a range holds at most 128 rows more than T / 512, the ranges are added after
    rows = min(T, 160)
    _close("dw_router", g["dw_router"], x64.T @ dl64, (6 * rows + 64) * U * (np.abs(x64).T @ np.abs(dl64)))
    if add:   # in place
        op.dx = add_dev
        assert torch.equal(op(*dev, dx_in=add_dev)["dx"], first["dx"])


@pytest.mark.parametrize("T, d, E", [(70001, 64, 20), (33100, 320, 33), (262300, 64, 9), (131100, 128, 64)])
@pytest.mark.parametrize("add", [False, True])
def test_router_backward_many_tokens(T, d, E, add):
    """Several tiles of tokens for a workgroup, the last of them short, and rows past 32 MB."""
    print(f"[router backward] T={T} d={d} E={E} add={add}", flush=True)
    g = torch.Generator().manual_seed(T)
    dl = torch.randn(T, E, generator=g)
    x, w, a = (torch.randn(*s, generator=g).to(torch.bfloat16) for s in ((T, d), (d, E), (T, d)))
    op = B.RouterBackward(B.problem(T, d, E, 1, 64, "bf16"), DEV)
    dev = [t.to(DEV) for t in (dl, x, w)]
    add_dev = a.to(DEV) if add else None
    first = {k: v.clone() for k, v in op(*dev, dx_in=add_dev).items()}
    dl64, x64, w64, a64 = (as_f64(t) for t in (dl, x, w, a))
    ref = dl64 @ w64.T + (a64 if add else 0)
    mag = np.abs(dl64) @ np.abs(w64).T + (np.abs(a64) if add else 0)
    _close("dx", first["dx"], ref, 2.0 ** -8 * np.abs(ref) + (6 * E + 16) * U * mag)
    # up to 512 ranges of T / 512 rows (rounded up by less than 160), added after
    _close("dw_router", first["dw_router"], x64.T @ dl64,
           (6 * (T / 512 + 160) + 512 + 64) * U * (np.abs(x64).T @ np.abs(dl64)))
    if add:   # in place
        op.dx = add_dev
        assert torch.equal(op(*dev, dx_in=add_dev)["dx"], first["dx"])
