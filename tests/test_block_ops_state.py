"""What the operators' objects keep from call to call, and calls that do not go
together: checked on the host (no GPU needed)."""
import ctypes

import pytest
import torch

from routing_dispatch_grouped_router_amd import binding as B

F = ctypes.c_void_p(0x1000)
G = ctypes.c_void_p(0x3000)


def _p(T=64, d=256, E=8, k=2, H=256, act="mxfp8", **kw):
    return B.problem(T, d, E, k, H, act, **kw)


@pytest.fixture
def accepting(monkeypatch):
    """A library that takes every call, for host tensors."""
    real, calls = B.lib(), []

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return getattr(real, name)
            return lambda *a: calls.append(name) or 0
    monkeypatch.setattr(B, "lib", lambda: Lib())
    monkeypatch.setattr(B, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(B, "_stream", lambda *a, **k: 0)
    return calls


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


def test_norm_of_a_sum_that_is_not_kept(accepting, monkeypatch):
    """sum is optional: nothing reads that of the last norm."""
    monkeypatch.setattr(B, "_inputs", lambda device, *t: [None if v is None else v.data_ptr() for v in t])
    x, w = torch.zeros(64, 256, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.bfloat16)
    op = B.Norm(_p(act="bf16"), "cpu")
    op.sum = None
    op(x, w, residual=x)
    op(x, w)                                                  # as before
    assert accepting == ["moe_norm"] * 2
    op = B.Norm(_p(act="bf16"), "cpu")
    with pytest.raises(ValueError, match="residual: expected"):
        op(x, w)
    op = B.Norm(_p(act="bf16"), "cpu", residual=False)
    with pytest.raises(ValueError, match="residual: not expected"):
        op(x, w, residual=x)
    op._index = x.get_device()
    monkeypatch.setattr(B, "_ptr", lambda t: t.data_ptr())
    op.sum = x.clone()
    op(x, w, residual=x)


@pytest.mark.parametrize("given", [False, True])
def test_backward_takes_the_codes_its_forward_took(accepting, given):
    p = _p(logits_given=given)
    fwd, bwd = B.Forward(p, "cpu"), B.Backward(p, "cpu", aux=True)
    x, w = torch.zeros(64, 256, dtype=torch.bfloat16), torch.zeros(256, 8, dtype=torch.bfloat16)
    q, qs = torch.zeros(64, 256, dtype=torch.uint8), torch.zeros(64, 8, dtype=torch.uint8)
    kw = dict(logits=torch.zeros(64, 8)) if given else dict(w_router=w)
    rows = dict(x=x, w_router=None if given else w)

    def back(**more):
        return bwd(fwd, x, None, w, **rows, **more)
    fwd(x, packed=w, xq=q, xq_scale=qs, **kw)
    del accepting[:]
    with pytest.raises(ValueError, match="xq"):
        back()
    with pytest.raises(ValueError, match="xq"):
        back(dlogits_aux=torch.zeros(64, 8))
    assert not accepting
    back(xq=q)
    back(xq=q.clone())                                        # the same codes kept elsewhere
    fwd(x, packed=w, **kw)
    del accepting[:]
    with pytest.raises(ValueError, match="xq"):
        back(xq=q)
    assert not accepting
    back()
    back(dlogits_aux=torch.zeros(64, 8))
    # a call that was refused leaves what the workspace holds
    fwd(x, packed=w, xq=q, xq_scale=qs, **kw)
    with pytest.raises(ValueError):
        fwd(x[:3], packed=w, **kw)
    back(xq=q)


def test_backward_of_a_forward_that_has_not_run(accepting):
    p = _p()
    fwd, bwd = B.Forward(p, "cpu"), B.Backward(p, "cpu")
    x, w = torch.zeros(64, 256, dtype=torch.bfloat16), torch.zeros(256, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="xq"):
        bwd(fwd, x, None, w, x=x, w_router=w, xq=torch.zeros(64, 256, dtype=torch.uint8))


def test_dx_over_x_is_refused_where_x_is_read_after_it():
    """dw_router is made from x after dx is written, in the dense gradient and in the sparse one."""
    for act, aux, xq in (("mxfp8", G, None), ("mxfp8", G, F), ("mxfp8", None, F), ("bf16", G, None), ("f32", G, None)):
        p, n = _p(act=act), ctypes.c_size_t()
        assert B.lib().moe_backward_aux_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == 0
        assert B.lib().moe_backward_aux(ctypes.byref(p), F, F, F, F, F, None, None, None, None, F, B.workspace_bytes(p), F,
                                        F, F, F, F, F, F, n.value, None, aux, xq) == -7
