"""Layer norm of rows whose values are all the same, at widths whose reciprocal times the row's total is not the value
(marked gpu)."""
import numpy as np
import pytest
import torch

from routing_dispatch_grouped_router_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
VALUES = [2.0 ** 50, 1e12, -4096.0, 3.7, 1e-20]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("d", [64, 1024, 3136, 4800, 6272, 10304, 16192])
def test_a_row_of_one_value_gives_the_bias(d, residual, bias, act):
    print(f"[constant rows] d={d} {act} residual={residual} bias={bias}", flush=True)
    rng = np.random.default_rng(d)
    dt, T = B.storage_dtype(act), len(VALUES)
    x = torch.tensor(VALUES).to(dt)[:, None].expand(T, d).contiguous().to(DEV)
    r = (2 * x[:, :1].float()).to(dt).expand(T, d).contiguous() if residual else None   # the sum is one value as well
    w, b = (torch.from_numpy(rng.standard_normal(d).astype(np.float32)).to(DEV).to(dt) for _ in range(2))
    op = B.LayerNorm(B.problem(T, d, 1, 1, 128, act), DEV, eps=1e-5, residual=residual)
    y = op(x, w, b if bias else None, residual=r)
    torch.cuda.synchronize()
    assert torch.equal(y, b.expand(T, d) if bias else torch.zeros_like(y))
    s = x[:, 0].float() if r is None else x[:, 0].float() + r[:, 0].float()
    assert torch.equal(op.mean, s)
    # the variance is 0: rstd is eps^-1/2, of the float32 eps, rounded once
    assert torch.equal(op.rstd.cpu(), torch.full((T,), float(np.float32(1) * np.float32(np.float64(np.float32(1e-5)) ** -0.5))))


def test_mxfp8_rows_of_one_value_are_zero():
    d = 6272
    x = torch.tensor(VALUES).bfloat16()[:, None].expand(len(VALUES), d).contiguous().to(DEV)
    op = B.LayerNorm(B.problem(len(VALUES), d, 1, 1, 128, "mxfp8"), DEV, residual=False)
    y = op(x, torch.ones(d, dtype=torch.bfloat16, device=DEV))
    torch.cuda.synchronize()
    assert not y.any() and not (op.q & 127).any()
