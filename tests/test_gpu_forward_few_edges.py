"""The block for a few tokens at the ends of its inputs' ranges (marked gpu): infinite and NaN logits choose as moe_route,
and MXFP8 weights whose blocks have the smallest scales."""
import numpy as np
import pytest
import torch

from routing_dispatch_grouped_router_amd import binding as B
from test_gpu_forward_few import Case

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("E, k", [(8, 3), (33, 4), (256, 8)])
def test_logits_that_are_not_finite(E, k):
    inf, nan = float("inf"), float("nan")
    c = Case(12, 128, E, k, 64, "bf16", given=True)
    for t, v in enumerate([[inf], [inf, inf, 1.0], [-inf] * E, [-inf] * (E - 1), [nan], [nan, inf, nan], [-nan], [0.0, -0.0] * 4,
                           [3e38, -3e38], [-inf, nan]]):
        c.logits[t, :len(v)] = torch.tensor(v[:E])
    c.dev["logits"].copy_(c.logits)
    c.run()
    r = B.route(c.p, logits=c.dev["logits"])
    torch.cuda.synchronize()
    assert torch.equal(r["idx"], c.op.idx)
    assert torch.allclose(r["gate"], c.op.gate, rtol=64 * U, atol=0, equal_nan=True)


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("size", [2.0 ** -118, 2.0 ** -124])
def test_weights_of_the_smallest_scales(size, T):
    """Blocks whose largest values need a scale of 2^-127: their codes times it, as everywhere."""
    c = Case(T, 256, 4, 2, 128, "mxfp8", given=True, scale=size)
    c.w[1] = (c.w[1].float() * 2.0 ** 60).to(torch.bfloat16)
    c.w[2] = (c.w[2].float() * 2.0 ** 100).to(torch.bfloat16)
    c.x = (c.x.float() * 2.0 ** 70).to(torch.bfloat16)
    c.dev["x"].copy_(c.x)
    c.packed.copy_(B.pack_weights(c.p, *(w.to("cuda:0") for w in c.w)))
    c.run()
    c.check()
    assert c.op.y.any()
