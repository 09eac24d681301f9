"""Layer norm (moe_layer_norm, moe_layer_norm_backward) against its float64 oracle (marked gpu).

Tolerances, from the arithmetic (u = 2^-24, half a float32 step; a stored value
is off by half a step of its type).  Forward: everything past the float32 sum s
is float64, so what is left is that sum's rounding (u |s|, where there is a
residual), which moves the mean by u mean|s| and, to first order, rstd by
u rms(s) rstd of it (1.01: the second order), and the roundings of the results.
Backward: float32 sums of d terms run over at most 128 terms per thread and a
tree of 8 (d <= 32768), and a result takes a handful of products: 160 u of the
sum of magnitudes bound every sum and what is made of it."""
import numpy as np
import pytest
import torch

from oracle import mxfp8 as MX
from oracle import training_ops as Q
from routing_dispatch_grouped_router_amd import binding as B
from routing_dispatch_grouped_router_amd.workloads import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "mxfp8": 2.0 ** -8}


def _rand(rng, shape, act, scale=1.0, mean=0.0):
    return torch.from_numpy((mean + scale * rng.standard_normal(shape)).astype(np.float32)).to(B.storage_dtype(act))


def _close(name, got, ref, tol):
    got = as_f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} values off, worst {np.max((np.abs(got - ref) - tol)):.3e}"


def _problem(T, d, act):
    return B.problem(T, d, 1, 1, 128, act)


def _check_forward(op, x, r, w, b, act, eps, y):
    s, mean, rstd, ref = Q.layer_norm(as_f64(x), None if r is None else as_f64(r), as_f64(w),
                                      None if b is None else as_f64(b), eps)
    off = U * np.abs(s) if r is not None else np.zeros_like(s)         # of s
    off_mean = off.mean(1)
    rel_rstd = 1.01 * np.sqrt((off ** 2).mean(1)) * rstd + 2.0 ** -45
    e = np.abs(s - mean[:, None])
    tol = np.abs(as_f64(w)) * rstd[:, None] * (off + off_mean[:, None] + e * rel_rstd[:, None]) + 2.0 ** -45 * np.abs(ref)
    _close("mean", op.mean, mean, U * np.abs(mean) + off_mean + 2.0 ** -45 * np.abs(s).mean(1))
    _close("rstd", op.rstd, rstd, (U + rel_rstd) * rstd)
    _close("y", y, ref, tol * 1.01 + (HALF[act] + 2 * U) * np.abs(ref))
    if r is not None:
        _close("sum", op.sum, s, (HALF[act] + 2 * U) * np.abs(s))


# one token, a few, counts around the tile sizes, widths of every register variant and beyond them
SHAPES = [(1, 64), (1, 4096), (3, 192), (5, 512), (130, 576), (1023, 1024), (1025, 2048), (2100, 4096), (70, 8192),
          (9, 16448), (2, 32768), (4200, 4096)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("T, d", SHAPES)
def test_layer_norm(T, d, act, residual):
    if act == "mxfp8":
        d = (d + 127) // 128 * 128
    print(f"[layer norm] T={T} d={d} {act} residual={residual}", flush=True)
    rng = np.random.default_rng(T * 7 + d)
    x = _rand(rng, (T, d), act, mean=0.5)
    x[rng.random((T, d)) < 0.01] *= 64
    r = _rand(rng, (T, d), act) if residual else None
    w, b = _rand(rng, (d,), act), _rand(rng, (d,), act) if T % 2 else None
    x[T // 2] = 0                                 # a row of zeros (of the residual alone)
    op = B.LayerNorm(_problem(T, d, act), DEV, eps=1e-5, residual=residual)
    for t in (op.y, op.sum, op.q, op.q_scale, op.mean, op.rstd):
        if t is not None:
            t.fill_(7)
    y = op(x.to(DEV), w.to(DEV), None if b is None else b.to(DEV), residual=None if r is None else r.to(DEV))
    torch.cuda.synchronize()
    _check_forward(op, x, r, w, b, act, 1e-5, y)
    if act == "mxfp8":   # the codes are exactly those of the stored rows
        codes, scales = MX.quantize(as_f64(y))
        assert np.array_equal(op.q.cpu().numpy(), codes) and np.array_equal(op.q_scale.cpu().numpy(), scales)
    else:
        assert op.q is None


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_rows_with_a_mean_far_from_zero(act):
    """What the mean leaves is kept: 2^12 times the spread, and a row whose values are all the same."""
    T, d = 40, 1024
    rng = np.random.default_rng(8)
    x = _rand(rng, (T, d), act, mean=4096.0)
    x[7] = 3.5
    w, b = _rand(rng, (d,), act), _rand(rng, (d,), act)
    op = B.LayerNorm(_problem(T, d, act), DEV, residual=False)
    y = op(x.to(DEV), w.to(DEV), b.to(DEV))
    _check_forward(op, x, None, w, b, act, 1e-5, y)
    assert torch.equal(y[7].cpu(), b)


@pytest.mark.parametrize("scale", [1e-30, 3e37])
def test_rows_at_the_ends_of_the_range(scale):
    """Squares outside float32's range: the norm of scaled rows is that of the rows."""
    T, d = 12, 512
    rng = np.random.default_rng(9)
    x, w = _rand(rng, (T, d), "f32", scale=scale), _rand(rng, (d,), "f32")
    x = x.clamp(-3e38, 3e38)
    op = B.LayerNorm(_problem(T, d, "f32"), DEV, residual=False, eps=0.0)
    y = op(x.to(DEV), w.to(DEV))
    _, mean, _, ref = Q.layer_norm(as_f64(x), None, as_f64(w), None, 0.0)
    _close("mean", op.mean, mean, U * np.abs(mean) + 2.0 ** -45 * np.abs(as_f64(x)).mean(1) + 2.0 ** -150)
    _close("y", y, ref, 3 * U * np.abs(ref))


# 512: a row in registers; 16512: rows read again; (4200, 4096): streamed past the caches
@pytest.mark.parametrize("T, d", [(300, 512), (5, 16512), (4200, 4096)])
def test_in_place_and_codes_only(T, d):
    rng = np.random.default_rng(1)
    x, r, w, b = (_rand(rng, s, "mxfp8").to(DEV) for s in ((T, d), (T, d), (d,), (d,)))
    op = B.LayerNorm(_problem(T, d, "mxfp8"), DEV)
    op(x, w, b, residual=r)
    want = [t.clone() for t in (op.sum, op.y, op.q, op.q_scale, op.mean, op.rstd)]
    x2, r2 = x.clone(), r.clone()             # sum over the residual, y over x
    op2 = B.LayerNorm(_problem(T, d, "mxfp8"), DEV)
    op2.sum, op2.y = r2, x2
    op2(x2, w, b, residual=r2)
    op3 = B.LayerNorm(_problem(T, d, "mxfp8"), DEV)   # no bf16 rows, and no sum
    op3.y = op3.sum = op3.mean = None
    op3(x, w, b, residual=r)
    torch.cuda.synchronize()
    for p, q in zip(want, (r2, x2, op2.q, op2.q_scale, op2.mean, op2.rstd)):
        assert torch.equal(p, q)
    assert torch.equal(op3.q, want[2]) and torch.equal(op3.q_scale, want[3]) and torch.equal(op3.rstd, want[5])


def test_rows_with_nonfinite_values_leave_the_others():
    T, d = 70, 256
    rng = np.random.default_rng(2)
    x, w = _rand(rng, (T, d), "bf16").to(DEV), _rand(rng, (d,), "bf16").to(DEV)
    op = B.LayerNorm(_problem(T, d, "bf16"), DEV, residual=False)
    want = op(x, w).clone()
    x[3, 5], x[40, 0] = float("nan"), float("inf")
    got = op(x, w)
    rows = [i for i in range(T) if i not in (3, 40)]
    assert torch.equal(got[rows], want[rows]) and got[3].isnan().all() and got[40].isnan().all()


BWD_SHAPES = [(1, 64), (1, 4096), (3, 192), (130, 576), (1000, 256), (777, 192), (2100, 1024), (5000, 128),
              (600, 4096), (70, 8192), (9, 16448), (700, 9216), (4200, 4096), (5, 32832), (300, 6144)]


@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T, d", BWD_SHAPES)
def test_layer_norm_backward(T, d, act, dsum):
    print(f"[layer norm backward] T={T} d={d} {act} dsum={dsum}", flush=True)
    rng = np.random.default_rng(T * 3 + d)
    s, dy, w = _rand(rng, (T, d), act, mean=0.5), _rand(rng, (T, d), act, 0.1), _rand(rng, (d,), act)
    s[rng.random((T, d)) < 0.01] *= 64
    ds_in = _rand(rng, (T, d), act, 0.1) if dsum else None
    _, mean, rstd, _ = Q.layer_norm(as_f64(s), None, as_f64(w), None, 1e-5)
    mean, rstd = (torch.from_numpy(v.astype(np.float32)) for v in (mean, rstd))
    op = B.LayerNormBackward(_problem(T, d, act), DEV)
    op.ws.fill_(255)
    dev = [t.to(DEV) for t in (dy, s, w, mean, rstd)]
    dsum_dev = None if ds_in is None else ds_in.to(DEV)
    g = op(*dev, dsum=dsum_dev)
    first = {k: v.clone() for k, v in g.items()}
    op(*dev, dsum=dsum_dev)
    torch.cuda.synchronize()
    assert all(torch.equal(first[k], g[k]) for k in g)
    s64, dy64, w64, m64, r64 = (as_f64(t) for t in (s, dy, w, mean, rstd))
    ds_ref, dw_ref, db_ref = Q.layer_norm_backward(dy64, None if ds_in is None else as_f64(ds_in), s64, w64, m64, r64)
    u, n = np.abs(dy64 * w64), np.abs((s64 - m64[:, None]) * r64[:, None])
    mag = r64[:, None] * (u + u.mean(1, keepdims=True) + n * (u * n).mean(1, keepdims=True))
    mag = mag + (0 if ds_in is None else np.abs(as_f64(ds_in)))
    _close("ds", g["ds"], ds_ref, HALF[act] * np.abs(ds_ref) + 160 * U * mag)
    # columns: T <= 5000 rows, at most 17 per thread, then 4 and 512 / 16 partial sums and 16 waves
    _close("dweight", g["dweight"], dw_ref, 80 * U * (np.abs(dy64) * n).sum(0))
    _close("dbias", g["dbias"], db_ref, 80 * U * np.abs(dy64).sum(0))
    # a norm without a bias: the other gradients as before
    op.dbias = None
    h = op(*dev, dsum=dsum_dev)
    assert h["dbias"] is None and torch.equal(h["ds"], first["ds"]) and torch.equal(h["dweight"], first["dweight"])


# a wave's rows, a workgroup's rows past the caches, wider ones, rows read twice
@pytest.mark.parametrize("T, d", [(500, 256), (4200, 4096), (40, 8448), (7, 16448)])
def test_layer_norm_backward_in_place(T, d):
    rng = np.random.default_rng(5)
    s, dy, e, w = (_rand(rng, sh, "bf16").to(DEV) for sh in ((T, d), (T, d), (T, d), (d,)))
    mean = s.float().mean(1)
    rstd = ((s.float() - mean[:, None]).square().mean(1) + 1e-6).rsqrt()
    op = B.LayerNormBackward(_problem(T, d, "bf16"), DEV)
    want = {k: v.clone() for k, v in op(dy, s, w, mean, rstd, dsum=e).items()}
    for target in ("dy", "dsum"):
        dy2, e2 = dy.clone(), e.clone()
        op.ds = dy2 if target == "dy" else e2
        g = op(dy2, s, w, mean, rstd, dsum=e2)
        assert all(torch.equal(g[k], want[k]) for k in want)
