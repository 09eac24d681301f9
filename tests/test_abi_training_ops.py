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
