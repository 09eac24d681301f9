"""The norm (moe_norm, moe_norm_backward) against its float64 oracle (marked gpu).

Tolerances, from the arithmetic: a stored value is off by half a step of its
type (bf16 2^-8, float32 2^-24 of it).  Float32 sums of d terms here run over
at most 128 terms per thread and a tree of 8 (d <= 32768), and a result takes
a handful of products: 160 half-steps (u = 2^-24) of the sum of magnitudes
bound every sum and what is made of it."""
import numpy as np
import pytest
import torch

from oracle import block_ops as Q
from oracle import mxfp8 as MX
from routing_dispatch_grouped_router_amd import binding as B
from routing_dispatch_grouped_router_amd.workloads import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "mxfp8": 2.0 ** -8}


def _rand(rng, shape, act, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(B.storage_dtype(act))


def _close(name, got, ref, tol):
    got, bad = as_f64(got), None
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{name}: {bad.sum()} values off, worst {np.max((np.abs(got - ref) - tol)):.3e}"


def _problem(T, d, act):
    return B.problem(T, d, 1, 1, 128, act)


# one token, a few, counts around the tile sizes, widths of every register variant and beyond them
SHAPES = [(1, 64), (1, 4096), (3, 192), (5, 512), (130, 576), (1023, 1024), (1025, 2048), (2100, 4096), (70, 8192),
          (9, 16448), (2, 32768), (4200, 4096)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("T, d", SHAPES)
def test_norm(T, d, act, residual):
    if act == "mxfp8":
        d = (d + 127) // 128 * 128
    print(f"[norm] T={T} d={d} {act} residual={residual}", flush=True)
    rng = np.random.default_rng(T * 7 + d)
    x = _rand(rng, (T, d), act)
    x[rng.random((T, d)) < 0.01] *= 64
    r = _rand(rng, (T, d), act) if residual else None
    w = _rand(rng, (d,), act)
    x[T // 2] = 0                                 # a row of zeros (of the residual alone)
    op = B.Norm(_problem(T, d, act), DEV, eps=1e-5, residual=residual)
    for t in (op.y, op.sum, op.q, op.q_scale, op.rstd):
        if t is not None:
            t.fill_(7)
    y = op(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV))
    torch.cuda.synchronize()
    s_ref, rstd_ref, y_ref = Q.rmsnorm(as_f64(x), None if r is None else as_f64(r), as_f64(w), 1e-5)
    _close("rstd", op.rstd, rstd_ref, 160 * U * rstd_ref)
    _close("y", y, y_ref, (HALF[act] * (1 + 160 * U) + 160 * U) * np.abs(y_ref))
    if residual:
        _close("sum", op.sum, s_ref, (HALF[act] + 2 * U) * np.abs(s_ref))
    if act == "mxfp8":   # the codes are exactly those of the stored rows
        codes, scales = MX.quantize(as_f64(y))
        assert np.array_equal(op.q.cpu().numpy(), codes) and np.array_equal(op.q_scale.cpu().numpy(), scales)
    else:
        assert op.q is None


# 512: a row in registers; 16512: rows read twice; (4200, 4096): streamed past the caches
@pytest.mark.parametrize("T, d", [(300, 512), (5, 16512), (4200, 4096)])
def test_norm_in_place_and_codes_only(T, d):
    rng = np.random.default_rng(1)
    x, r, w = (_rand(rng, s, "mxfp8").to(DEV) for s in ((T, d), (T, d), (d,)))
    op = B.Norm(_problem(T, d, "mxfp8"), DEV)
    op(x, w, residual=r)
    want = [t.clone() for t in (op.sum, op.y, op.q, op.q_scale, op.rstd)]
    # sum over the residual, y over x
    x2, r2 = x.clone(), r.clone()
    op2 = B.Norm(_problem(T, d, "mxfp8"), DEV)
    op2.sum, op2.y = r2, x2
    op2(x2, w, residual=r2)
    # no bf16 rows
    op3 = B.Norm(_problem(T, d, "mxfp8"), DEV)
    op3.y = None
    op3(x, w, residual=r)
    torch.cuda.synchronize()
    for a, b in zip(want, (r2, x2, op2.q, op2.q_scale, op2.rstd)):
        assert torch.equal(a, b)
    assert torch.equal(op3.q, want[2]) and torch.equal(op3.q_scale, want[3])


def test_norm_of_rows_with_nonfinite_values_leaves_the_others():
    T, d = 70, 256
    rng = np.random.default_rng(2)
    x, w = _rand(rng, (T, d), "bf16").to(DEV), _rand(rng, (d,), "bf16").to(DEV)
    op = B.Norm(_problem(T, d, "bf16"), DEV, residual=False)
    want = op(x, w).clone()
    x[3, 5], x[40, 0] = float("nan"), float("inf")
    got = op(x, w)
    rows = [i for i in range(T) if i not in (3, 40)]
    assert torch.equal(got[rows], want[rows]) and got[3].isnan().all()


BWD_SHAPES = [(1, 64), (1, 4096), (3, 192), (130, 576), (1000, 256), (2100, 1024), (5000, 128), (600, 4096), (70, 8192),
              (9, 16448), (700, 9216), (4200, 4096)]


@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T, d", BWD_SHAPES)
def test_norm_backward(T, d, act, dsum):
    print(f"[norm backward] T={T} d={d} {act} dsum={dsum}", flush=True)
    rng = np.random.default_rng(T * 3 + d)
    s, dy, w = _rand(rng, (T, d), act), _rand(rng, (T, d), act, 0.1), _rand(rng, (d,), act)
    s[rng.random((T, d)) < 0.01] *= 64
    ds_in = _rand(rng, (T, d), act, 0.1) if dsum else None
    rstd = torch.from_numpy((1 / np.sqrt((as_f64(s) ** 2).mean(1) + 1e-5)).astype(np.float32))
    op = B.NormBackward(_problem(T, d, act), DEV)
    op.ws.fill_(255)
    dev = [t.to(DEV) for t in (dy, s, w, rstd)]
    dsum_dev = None if ds_in is None else ds_in.to(DEV)
    g = op(*dev, dsum=dsum_dev)
    first = {k: v.clone() for k, v in g.items()}
    op(*dev, dsum=dsum_dev)
    torch.cuda.synchronize()
    assert all(torch.equal(first[k], g[k]) for k in g)
    s64, dy64, w64, r64 = (as_f64(t) for t in (s, dy, w, rstd))
    ds_ref, dw_ref = Q.rmsnorm_backward(dy64, None if ds_in is None else as_f64(ds_in), s64, w64, rstd=r64)
    u, n = np.abs(dy64 * w64), np.abs(s64 * r64[:, None])
    mag = r64[:, None] * (u + n * (u * n).mean(1, keepdims=True)) + (0 if ds_in is None else np.abs(as_f64(ds_in)))
    _close("ds", g["ds"], ds_ref, HALF[act] * np.abs(ds_ref) + 160 * U * mag)
    # the weight gradient: T <= 5000 rows, at most 17 per thread, then 4 and 512 / 16 partial sums and 16 waves
    _close("dweight", g["dweight"], dw_ref, 80 * U * (np.abs(dy64) * n).sum(0))


# a wave's rows, a workgroup's rows past the caches, rows read twice
@pytest.mark.parametrize("T, d", [(500, 256), (4200, 4096), (40, 8448)])
def test_norm_backward_in_place(T, d):
    rng = np.random.default_rng(5)
    s, dy, e, w = (_rand(rng, sh, "bf16").to(DEV) for sh in ((T, d), (T, d), (T, d), (d,)))
    rstd = (s.float().square().mean(1) + 1e-6).rsqrt()
    op = B.NormBackward(_problem(T, d, "bf16"), DEV)
    want = {k: v.clone() for k, v in op(dy, s, w, rstd, dsum=e).items()}
    for target in ("dy", "dsum"):
        dy2, e2 = dy.clone(), e.clone()
        op.ds = dy2 if target == "dy" else e2
        g = op(dy2, s, w, rstd, dsum=e2)
        assert torch.equal(g["ds"], want["ds"]) and torch.equal(g["dweight"], want["dweight"])
