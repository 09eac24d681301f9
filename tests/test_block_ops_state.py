"""What the operators' objects keep from call to call: checked on the host (no
GPU needed)."""
import pytest
import torch

from routing_dispatch_grouped_router_amd import binding as B


def _p(T=64, d=256, E=8, k=2, H=256, act="mxfp8", **kw):
    return B.problem(T, d, E, k, H, act, **kw)


def test_counts_follow_the_buffer_put_in_place(monkeypatch):
    op = B.BalanceLoss(_p(act="f32"), "cpu")
    monkeypatch.setattr(B, "_ptr", lambda t: t.data_ptr())
    other = torch.arange(9, dtype=torch.int32)
    op._index = other.get_device()
    op.counts_live = other
    assert op.counts.data_ptr() == other.data_ptr() and op.counts.tolist() == list(range(8))
    assert op.live.tolist() == [8]
    for name in ("counts", "live"):                           # parts of counts_live, not buffers
        with pytest.raises(AttributeError):
            setattr(op, name, other[:1])
