"""AdamW over parameters that require gradients (marked gpu): masters made from them are plain tensors."""
import copy

import pytest
import torch

from routing_dispatch_grouped_router_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_masters_of_parameters_are_no_part_of_a_graph():
    w = [torch.nn.Parameter(torch.randn(300, device=DEV).bfloat16()), torch.nn.Parameter(torch.randn(7, device=DEV))]
    g = [torch.randn(300, device=DEV), torch.randn(7, device=DEV)]
    op = B.AdamW(w, g, lr=0.01, master=True)
    assert op.master[1] is None and op.master[0].dtype == torch.float32
    assert not op.master[0].requires_grad and op.master[0].grad_fn is None
    start = copy.deepcopy(op.master)               # a checkpoint's copy: refused for a tensor within a graph
    assert torch.equal(start[0], w[0].detach().float())
    op()
    torch.cuda.synchronize()
    assert not torch.equal(op.master[0], start[0]) and torch.equal(w[0].detach(), op.master[0].bfloat16())
    assert op.step.tolist() == [1, 0]
