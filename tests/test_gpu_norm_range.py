"""The norm over the whole range of its types (marked gpu): every value held to
the float64 oracle, NaN or an unwritten output among them counted as wrong;
rows whose squares leave float32's range; y to the last float32 bit.

A stored value is off by half a step of its type (bf16 2^-8, float32 2^-24 of
it); 160 half-steps (u = 2^-24) bound what float32 arithmetic adds."""
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
# a wave's rows of one and two chunks a lane, a workgroup's of one, two and four, rows read twice, rows past the caches
SHAPES = [(1, 64), (5, 512), (130, 576), (37, 1024), (21, 2048), (9, 4096), (70, 8192), (3, 16512), (4200, 4096)]


def _rand(rng, shape, act, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(B.storage_dtype(act))


def _close(name, got, ref, tol):
    bad = ~(np.abs(as_f64(got) - ref) <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} values off"


def _d(d, act):
    return (d + 127) // 128 * 128 if act == "mxfp8" else d


def _norm(x, w, r, act, eps):
    T, d = x.shape
    op = B.Norm(B.problem(T, d, 1, 1, 128, act), DEV, eps=eps, residual=r is not None)
    for t in (op.y, op.sum, op.rstd):
        if t is not None:
            t.fill_(float("nan"))
    op(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV))
    return op


def _check(op, x, w, r, act, eps):
    s, rstd, y = Q.rmsnorm(as_f64(x), None if r is None else as_f64(r), as_f64(w), eps)
    _close("rstd", op.rstd, rstd, 160 * U * rstd + 2.0 ** -149)
    # the last term: half a step of the type's subnormal values
    _close("y", op.y, y, (HALF[act] + 160 * U) * np.abs(y) + (2.0 ** -150 if act == "f32" else 2.0 ** -134))
    if r is not None:
        _close("sum", op.sum, s, (HALF[act] + 2 * U) * np.abs(s) + (2.0 ** -150 if act == "f32" else 2.0 ** -134))


@pytest.mark.parametrize("act", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T, d", SHAPES)
def test_every_value_is_written_and_right(T, d, act, residual):
    d = _d(d, act)
    print(f"[norm range] T={T} d={d} {act} residual={residual}", flush=True)
    rng = np.random.default_rng(T + d)
    x, w = _rand(rng, (T, d), act), _rand(rng, (d,), act)
    r = _rand(rng, (T, d), act) if residual else None
    _check(_norm(x, w, r, act, 1e-5), x, w, r, act, 1e-5)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("T, d", SHAPES)
def test_every_gradient_is_written_and_right(T, d, act, dsum):
    print(f"[norm backward range] T={T} d={d} {act} dsum={dsum}", flush=True)
    rng = np.random.default_rng(T * 3 + d)
    s, dy, w = _rand(rng, (T, d), act), _rand(rng, (T, d), act, 0.1), _rand(rng, (d,), act)
    e = _rand(rng, (T, d), act, 0.1) if dsum else None
    rstd = torch.from_numpy((1 / np.sqrt((as_f64(s) ** 2).mean(1) + 1e-5)).astype(np.float32))
    op = B.NormBackward(B.problem(T, d, 1, 1, 128, act), DEV)
    op.ws.fill_(255)
    op.ds.fill_(float("nan"))
    op.dweight.fill_(float("nan"))
    g = op(*(t.to(DEV) for t in (dy, s, w, rstd)), dsum=None if e is None else e.to(DEV))
    s64, dy64, w64, r64 = (as_f64(t) for t in (s, dy, w, rstd))
    ds, dw = Q.rmsnorm_backward(dy64, None if e is None else as_f64(e), s64, w64, rstd=r64)
    u, n = np.abs(dy64 * w64), np.abs(s64 * r64[:, None])
    mag = r64[:, None] * (u + n * (u * n).mean(1, keepdims=True)) + (0 if e is None else np.abs(as_f64(e)))
    _close("ds", g["ds"], ds, HALF[act] * np.abs(ds) + 160 * U * mag)
    # at most 17 rows per thread, then 4 and 512 / 16 partial sums and 16 waves
    _close("dweight", g["dweight"], dw, 80 * U * (np.abs(dy64) * n).sum(0))


# around the powers at which a square, or the mean of squares, leaves float32's range, and at the ends of its values
POWERS = [-126, -120, -80, -75, -64, -63, -60, 60, 63, 64, 80, 120, 126]


@pytest.mark.parametrize("act", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("d", [64, 1024, 4096, 16512])
def test_rows_whose_squares_leave_float32s_range(d, residual, act):
    d = _d(d, act)
    rng = np.random.default_rng(d)
    T = len(POWERS) + 2
    scale = 2.0 ** np.array([*POWERS, 0, 0])[:, None]
    x = torch.from_numpy(scale * (0.25 + 0.25 * rng.random((T, d))) * rng.choice([-1.0, 1.0], (T, d)))
    r = torch.from_numpy(scale * (0.25 + 0.25 * rng.random((T, d)))).to(B.storage_dtype(act)) if residual else None
    x = x.to(B.storage_dtype(act))
    x[-1, d // 2] = 2.0 ** 100                                # one value that leaves the others next to nothing
    w = _rand(rng, (d,), act)
    op = _norm(x, w, r, act, 0.0)
    _check(op, x, w, r, act, 0.0)
    if act == "mxfp8":
        codes, scales = MX.quantize(as_f64(op.y))
        assert np.array_equal(op.q.cpu().numpy(), codes) and np.array_equal(op.q_scale.cpu().numpy(), scales)


def test_subnormal_rows_and_rows_past_rstds_range():
    """Values below 2^-126: y is as always, rstd past float32's largest value infinite."""
    rng = np.random.default_rng(3)
    power = np.array([-127, -130, -140, -149])
    x = torch.from_numpy(2.0 ** power[:, None] * rng.integers(1, 4, (4, 512)) * rng.choice([-1.0, 1.0], (4, 512))).float()
    w = _rand(rng, (512,), "f32")
    op = _norm(x, w, None, "f32", 0.0)
    _, rstd, y = Q.rmsnorm(as_f64(x), None, as_f64(w), 0.0)
    _close("y", op.y, y, (HALF["f32"] + 160 * U) * np.abs(y))
    got, inside = as_f64(op.rstd), rstd < np.finfo(np.float32).max
    assert inside.any() and not inside.all() and np.isinf(got[~inside]).all()
    assert np.all(np.abs(got[inside] - rstd[inside]) <= 160 * U * rstd[inside])


def test_a_row_of_zeros_without_eps_has_no_norm():
    x, w = torch.zeros((3, 256), dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    x[1] = 2.0
    op = _norm(x, w, None, "bf16", 0.0)
    assert op.y[[0, 2]].isnan().all() and op.rstd[[0, 2]].isinf().all()
    assert torch.equal(op.y[1].cpu(), torch.ones(256, dtype=torch.bfloat16))


@pytest.mark.parametrize("act", ["bf16", "mxfp8", "f32"])
@pytest.mark.parametrize("T, d", [(8000, 512), (2000, 2048), (500, 8192), (250, 16512)])
def test_y_is_the_float32_nearest_for_the_float32_sum(T, d, act):
    """Residuals so far below x that the sum is rounded: y is the float32 next to the exact value for the rounded sum,
    rounded to its type; where 2^-40 of it decide, either."""
    print(f"[norm nearest] T={T} d={d} {act}", flush=True)
    rng = np.random.default_rng(T)
    x = _rand(rng, (T, d), act)
    r = (_rand(rng, (T, d), "f32") * torch.from_numpy(2.0 ** rng.integers(-20, -10, (T, d))).float()).to(x.dtype)
    w = _rand(rng, (d,), act)
    op = _norm(x, w, r, act, 1e-6)
    s = as_f64(x.float() + r.float())
    assert (s != as_f64(x) + as_f64(r)).mean() > 0.1
    _, _, y = Q.rmsnorm(s, None, as_f64(w), 1e-6)
    lo, hi = (torch.from_numpy((y * f).astype(np.float32)).to(x.dtype) for f in (1 - 2.0 ** -40, 1 + 2.0 ** -40))
    got = op.y.cpu()
    wrong = (got != lo) & (got != hi)
    assert not wrong.any(), f"{int(wrong.sum())} of {y.size} values"
    if act == "mxfp8":
        codes, scales = MX.quantize(as_f64(op.y))
        assert np.array_equal(op.q.cpu().numpy(), codes) and np.array_equal(op.q_scale.cpu().numpy(), scales)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_an_infinity_leaves_its_row_zeros_and_a_nan(residual, act):
    rng = np.random.default_rng(6)
    x, w = _rand(rng, (5, 1024), act), torch.ones(1024).to(B.storage_dtype(act))
    r = _rand(rng, (5, 1024), act) if residual else None
    good = _norm(x, w, r, act, 1e-6).y.clone()
    x[2, 7] = -float("inf")
    if residual:
        r[3, 9] = float("inf")
        x[4, 0], r[4, 0] = float("inf"), -float("inf")
    op = _norm(x, w, r, act, 1e-6)
    y = op.y.clone()
    assert torch.equal(y[:2], good[:2]) and op.rstd[2] == 0 and y[2, 7].isnan() and int((y[2] != 0).sum()) == 1
    if residual:
        assert op.rstd[3] == 0 and y[3, 9].isnan() and int((y[3] != 0).sum()) == 1 and op.sum[3, 9].isinf()
        assert y[4].isnan().all()


@pytest.mark.parametrize("T, d", [(130, 576), (21, 2048), (3, 16512), (4200, 4096)])
def test_a_sum_that_is_not_kept(T, d):
    rng = np.random.default_rng(4)
    x, r, w = (_rand(rng, sh, "bf16").to(DEV) for sh in ((T, d), (T, d), (d,)))
    op = B.Norm(B.problem(T, d, 1, 1, 128, "bf16"), DEV)
    y, rstd = op(x, w, residual=r).clone(), op.rstd.clone()
    op.sum = None
    assert torch.equal(op(x, w, residual=r), y) and torch.equal(op.rstd, rstd)
