"""Refusals of layer norm, the gradients' norm, the AdamW step and the block for
a few tokens: arguments are checked on the host, nothing is enqueued (no GPU
needed; the pointers are never followed)."""
import ctypes

import pytest
import torch

from routing_dispatch_grouped_router_amd import binding as B

F = ctypes.c_void_p(0x1000)
G = ctypes.c_void_p(0x2000)
ODD = ctypes.c_void_p(0x1004)
BIG = 1 << 40


def _p(T=64, d=256, E=8, k=2, H=256, act="bf16", **kw):
    return B.problem(T, d, E, k, H, act, **kw)


def _call(name, p, *args):
    return getattr(B.lib(), name)(ctypes.byref(p), *args)


def _swap(args, i, v):
    return [*args[:i], v, *args[i + 1:]]


def _query(name, p):
    n = ctypes.c_size_t()
    assert _call(name, p, ctypes.byref(n)) == 0
    assert n.value % 256 == 0
    assert _call(name, p, None) == -1
    assert getattr(B.lib(), name)(None, ctypes.byref(n)) == -1
    return n.value


def test_layer_norm():
    # x, residual, weight, bias, eps, sum, y, yq, yq_scale, mean, rstd, stream
    ok = [F, F, F, F, 1e-6, F, G, None, None, F, F, None]
    name = "moe_layer_norm"
    for act in ("bf16", "f32"):
        assert _call(name, _p(act=act), *_swap(_swap(ok, 7, F), 8, F)) == -3     # codes of a bf16 / f32 problem
    mx = _p(act="mxfp8")
    for i in (0, 2):
        assert _call(name, mx, *_swap(ok, i, None)) == -1
    assert _call(name, mx, *_swap(ok, 6, None)) == -1                            # neither y nor codes
    assert _call(name, mx, *_swap(ok, 7, F)) == -1                               # codes without scales
    for i in (0, 1, 2, 3, 5, 6):
        assert _call(name, mx, *_swap(ok, i, ODD)) == -7
    for i in (9, 10):
        assert _call(name, mx, *_swap(ok, i, ctypes.c_void_p(0x1002))) == -7
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _call(name, mx, *_swap(ok, 4, eps)) == -7
    assert _call(name, mx, *_swap(ok, 6, F)) == -7                               # y is sum
    assert _call(name, mx, *_swap(_swap(ok, 7, ODD), 8, F)) == -7
    assert _call(name, _p(T=0), *ok) == -2
    assert _call(name, _p(act="mxfp8", d=192), *ok) == -2


def test_layer_norm_backward():
    _query("moe_layer_norm_backward_workspace_bytes", _p())
    # dy, dsum, s, weight, mean, rstd, ds, dweight, dbias, ws, ws_bytes, stream
    ok = [F, F, F, F, F, F, G, F, F, F, BIG, None]
    name = "moe_layer_norm_backward"
    for i in (0, 2, 3, 4, 5, 6, 7, 9):
        assert _call(name, _p(), *_swap(ok, i, None)) == -1
    for i in (0, 1, 2, 3, 6, 7, 8, 9):
        assert _call(name, _p(), *_swap(ok, i, ODD)) == -7
    for i in (4, 5):
        assert _call(name, _p(), *_swap(ok, i, ctypes.c_void_p(0x1002))) == -7
    assert _call(name, _p(), *_swap(ok, 6, F)) == -7                             # ds is s
    assert _call(name, _p(), *_swap(ok, 10, 0)) == -4
    assert _call(name, _p(k=9), *ok) == -2


def test_layer_norm_binding(monkeypatch):
    monkeypatch.setattr(B, "_inputs", lambda device, *t: [None if v is None else v.data_ptr() for v in t])
    op = B.LayerNorm(_p(), "cpu")
    x, w = torch.zeros(64, 256, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.bfloat16)
    for args, kw, match in (((x, w), {}, "residual: expected"), ((x[:3], w), dict(residual=x), "x: expected"),
                            ((x, w.float()), dict(residual=x), "weight"), ((x, w, w[:5]), dict(residual=x), "bias"),
                            ((x, w), dict(residual=x.float()), "residual")):
        with pytest.raises(ValueError, match=match):
            op(*args, **kw)
    with pytest.raises(ValueError, match="residual: not expected"):
        B.LayerNorm(_p(), "cpu", residual=False)(x, w, residual=x)


def _param(**kw):
    base = dict(weight=0x10000, grad=0x20000, m=0x30000, v=0x40000, n=100, w_dtype=0, g_dtype=0, lr_scale=1.0, weight_decay=0.1)
    return B.Param(**{**base, **kw})


def _table(*params):
    arr, n, plan = (B.Param * max(1, len(params)))(*params), ctypes.c_size_t(), B.ParamPlan()
    st = B.lib().moe_param_table_bytes(arr, len(params), ctypes.byref(n))
    if st:
        return st, None, None
    assert n.value % 256 == 0
    buf = (ctypes.c_uint8 * n.value)()
    assert B.lib().moe_param_table(arr, len(params), buf, n.value - 1, ctypes.byref(plan)) == -4
    assert B.lib().moe_param_table(arr, len(params), None, n.value, ctypes.byref(plan)) == -1
    assert B.lib().moe_param_table(arr, len(params), buf, n.value, None) == -1
    return B.lib().moe_param_table(arr, len(params), buf, n.value, ctypes.byref(plan)), plan, buf


def test_param_table():
    assert B.lib().moe_param_table_bytes(None, 1, ctypes.byref(ctypes.c_size_t())) == -1
    assert _table()[0] == -2
    st, plan, _ = _table(_param())
    assert st == 0 and list(plan.first) == [0] + [1] * 13
    for kw, want in ((dict(grad=None), -1), (dict(m=None), -1), (dict(v=None), -1), (dict(m_scale=0x50000), -1),
                     (dict(weight=None), -1), (dict(n=-1), -2), (dict(n=1 << 38), -2), (dict(w_dtype=2), -3),
                     (dict(g_dtype=7), -3), (dict(master=0x60000), -3), (dict(lr_scale=float("nan")), -7),
                     (dict(weight_decay=float("inf")), -7)):
        assert _table(_param(**kw))[0] == want, kw
    for name in ("weight", "grad", "m", "v"):
        assert _table(_param(**{name: 0x70004}))[0] == -7
    assert _table(_param(m_scale=0x50002, v_scale=0x60000))[0] == -7
    assert _table(_param(m_scale=0x50004, v_scale=0x60000))[0] == 0
    # tensors that a step writes and others: 100 float32 are 400 bytes
    for name in ("grad", "m", "v"):
        assert _table(_param(**{name: 0x10000 + 384}))[0] == -7
        assert _table(_param(**{name: 0x10000 + 400}))[0] == 0
    assert _table(_param(weight=0x20000 - 384))[0] == -7
    assert _table(_param(), _param(weight=0x50000, m=0x60000, v=0x70000))[0] == 0        # one gradient of two
    assert _table(_param(), _param())[0] == -7
    assert _table(_param(w_dtype=1, master=0x50000, m_scale=0x60000, v_scale=0x60000))[0] == -7
    # kinds: float32; bf16 with a master; bf16 with 8-bit moments and bf16 gradient; a gradient alone; nothing
    st, plan, _ = _table(_param(n=5000), _param(w_dtype=1, master=0x150000, weight=0x110000, m=0x130000, v=0x140000),
                         _param(w_dtype=1, g_dtype=1, weight=0x210000, m=0x230000, v=0x240000, m_scale=0x250000, v_scale=0x260000, n=8193),
                         _param(weight=None, m=None, v=None), _param(n=0, weight=0, grad=0, m=0, v=0))
    assert st == 0 and list(plan.first) == [0] + [3] * 4 + [4] * 7 + [9, 10]
    assert _table(_param(n=(1 << 38) - 1), *[_param(weight=None, m=None, v=None, n=(1 << 38) - 1)] * 32)[0] == -2   # chunks


def test_grad_norm_and_adamw():
    _, plan, _ = _table(_param())
    _, alone, _ = _table(_param(weight=None, m=None, v=None))
    L, hyper = B.lib(), B.AdamwHyper(0.9, 0.999, 1e-8, 0)
    ref = ctypes.byref
    assert L.moe_grad_norm(None, F, 1.0, F, None) == -1 and L.moe_grad_norm(ref(plan), None, 1.0, F, None) == -1
    assert L.moe_grad_norm(ref(plan), F, 1.0, None, None) == -1 and L.moe_grad_norm(ref(B.ParamPlan()), F, 1.0, F, None) == -6
    for most in (0.0, -1.0, float("nan")):
        assert L.moe_grad_norm(ref(plan), F, most, F, None) == -7
    assert L.moe_grad_norm(ref(plan), ODD, 1.0, F, None) == -7
    assert L.moe_grad_norm(ref(plan), F, 1.0, ctypes.c_void_p(0x1001), None) == -7
    # plan, table, hyper, lr, clip, step, stream
    ok = [ref(plan), F, ref(hyper), F, None, F, None]
    for i in (0, 1, 2, 3, 5):
        assert L.moe_adamw(*_swap(ok, i, None)) == -1
    assert L.moe_adamw(*_swap(ok, 0, ref(alone))) == -6 and L.moe_adamw(*_swap(ok, 0, ref(B.ParamPlan()))) == -6
    for h in ((1.0, 0.9, 1e-8), (0.9, 1.0, 1e-8), (-0.1, 0.9, 1e-8), (0.9, float("nan"), 1e-8), (0.9, 0.9, -1.0), (0.9, 0.9, float("inf"))):
        assert L.moe_adamw(*_swap(ok, 2, ref(B.AdamwHyper(*h, 0)))) == -7
    assert L.moe_adamw(*_swap(ok, 1, ODD)) == -7
    for i in (3, 4, 5):
        assert L.moe_adamw(*_swap(ok, i, ctypes.c_void_p(0x1002))) == -7


def test_adamw_binding():
    w = torch.zeros(10)
    for args, kw, match in ((([], []), {}, "as many grads"), (([w], []), {}, "as many grads"), (([w], [w]), dict(states="4bit"), "states"),
                            (([w], [w]), dict(states="8bit", v=[w]), "8-bit states"), (([w], [w]), dict(m=[w[:3]]), "m: expected"),
                            (([w], [w]), dict(master=[None, None]), "master"), (([w], [w]), dict(weight_decay=[1.0, 2.0]), "weight_decay"),
                            (([w], [w]), dict(lr=torch.zeros(2)), "lr"), (([w], [w]), dict(step=torch.zeros(2)), "step")):
        with pytest.raises(ValueError, match=match):
            B.AdamW(*args, **kw)
    # iterators are read once: the only objection left is that the tensors are the host's
    with pytest.raises(ValueError, match="device tensor"):
        B.AdamW(iter([w]), iter([w]))
    with pytest.raises(ValueError, match="at least one"):
        B.GradNorm([])
    with pytest.raises(ValueError, match="device tensor"):
        B.GradNorm([w])


def test_forward_few():
    name = "moe_forward_few"
    _query(name + "_workspace_bytes", _p(T=32))
    # x, w_router, logits, packed, mask, y, idx, gate, ws, ws_bytes, stream
    ok = [F, F, F, F, None, G, None, None, F, BIG, None]
    p, given = _p(T=8), _p(T=8, logits_given=True)
    for i in (0, 1, 2, 3, 5, 8):
        assert _call(name, p, *_swap(ok, i, None)) == -1
    for i in (0, 2, 3, 5, 8):
        assert _call(name, given, *_swap(_swap(ok, 1, None), i, None)) == -1
    for i in (0, 1, 2, 3, 5, 8):
        assert _call(name, p, *_swap(ok, i, ODD)) == -7
    for i in (6, 7):
        assert _call(name, p, *_swap(ok, i, ctypes.c_void_p(0x1002))) == -7
    assert _call(name, p, *_swap(ok, 9, 64)) == -4
    assert _call(name, _p(T=33), *ok) == -2 and _call(name, _p(T=8, d=96), *ok) == -2
    assert _call(name, _p(T=8, act="mxfp8", H=192), *ok) == -2
    assert _call(name, _p(T=8, identity=True), *ok) == -3


def test_forward_few_binding(monkeypatch):
    monkeypatch.setattr(B, "_inputs", lambda device, *t: [None if v is None else v.data_ptr() for v in t])
    op = B.ForwardFew(_p(T=4), "cpu")
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(256, 8, dtype=torch.bfloat16)
    packed = torch.zeros(op.weight_bytes, dtype=torch.uint8)
    for args, kw, match in (((x[:3], packed), dict(w_router=w), "x: expected"), ((x, packed[:5]), dict(w_router=w), "packed"),
                            ((x, packed), {}, "w_router"), ((x, packed), dict(w_router=w, mask=torch.zeros(4)), "mask")):
        with pytest.raises(ValueError, match=match):
            op(*args, **kw)
    with pytest.raises(ValueError, match="logits"):
        B.ForwardFew(_p(T=4, logits_given=True), "cpu")(x, packed)
