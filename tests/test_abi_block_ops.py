"""Refusals of the operators around the block: arguments are checked on the
host, nothing is enqueued (no GPU needed; the pointers are never followed)."""
import ctypes

import pytest
import torch

from routing_dispatch_grouped_router_amd import binding as B

F = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1004)
BIG = 1 << 40


def _p(T=64, d=256, E=8, k=2, H=256, act="bf16", **kw):
    return B.problem(T, d, E, k, H, act, **kw)


def _call(name, p, *args):
    return getattr(B.lib(), name)(ctypes.byref(p), *args)


def _swap(args, i, v):
    return [*args[:i], v, *args[i + 1:]]


QUERIES = ["moe_norm_backward_workspace_bytes", "moe_balance_workspace_bytes", "moe_router_backward_workspace_bytes",
           "moe_backward_aux_workspace_bytes", "moe_decode_weight_bytes", "moe_decode_workspace_bytes"]


@pytest.mark.parametrize("name", QUERIES)
def test_queries(name):
    n = ctypes.c_size_t()
    assert _call(name, _p(), ctypes.byref(n)) == 0
    assert n.value % 256 == 0
    assert _call(name, _p(), None) == -1
    assert _call(name, _p(T=0), ctypes.byref(n)) == -2
    assert _call(name, _p(d=96), ctypes.byref(n)) == -2
    assert getattr(B.lib(), name)(None, ctypes.byref(n)) == -1


def test_norm():
    # x, residual, weight, eps, sum, y, yq, yq_scale, rstd, stream
    ok = [F, F, F, 1e-6, F, ctypes.c_void_p(0x2000), None, None, F, None]
    for act in ("bf16", "f32"):
        assert _call("moe_norm", _p(act=act), *_swap(_swap(ok, 6, F), 7, F)) == -3     # codes of a bf16 / f32 problem
    mx = _p(act="mxfp8")
    for i, st in [(0, -1), (2, -1)]:
        assert _call("moe_norm", mx, *_swap(ok, i, None)) == st
    assert _call("moe_norm", mx, *_swap(ok, 5, None)) == -1                            # neither y nor codes
    assert _call("moe_norm", mx, *_swap(ok, 6, F)) == -1                               # codes without scales
    for i in (0, 1, 2, 4, 5):
        assert _call("moe_norm", mx, *_swap(ok, i, ODD)) == -7
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _call("moe_norm", mx, *_swap(ok, 3, eps)) == -7
    assert _call("moe_norm", mx, *_swap(ok, 5, F)) == -7                               # y is sum
    assert _call("moe_norm", mx, *_swap(_swap(ok, 6, ODD), 7, F)) == -7
    assert _call("moe_norm", _p(T=0), *ok) == -2
    assert _call("moe_norm", _p(act="mxfp8", d=192), *ok) == -2


def test_norm_backward():
    # dy, dsum, s, weight, rstd, ds, dweight, ws, ws_bytes, stream
    ok = [F, F, F, F, F, ctypes.c_void_p(0x2000), F, F, BIG, None]
    for i in (0, 2, 3, 4, 5, 6, 7):
        assert _call("moe_norm_backward", _p(), *_swap(ok, i, None)) == -1
    for i in (0, 1, 2, 3, 5, 7):
        assert _call("moe_norm_backward", _p(), *_swap(ok, i, ODD)) == -7
    assert _call("moe_norm_backward", _p(), *_swap(ok, 5, F)) == -7                    # ds is s
    assert _call("moe_norm_backward", _p(), *_swap(ok, 8, 0)) == -4
    assert _call("moe_norm_backward", _p(k=9), *ok) == -2


def test_balance():
    # logits, topk_idx, mask, counts, loss, ws, ws_bytes, stream
    ok = [F, F, None, F, F, F, BIG, None]
    for i in (0, 1, 3, 4, 5):
        assert _call("moe_balance_loss", _p(), *_swap(ok, i, None)) == -1
    assert _call("moe_balance_loss", _p(), *_swap(ok, 6, 8)) == -4
    for i in (0, 5):
        assert _call("moe_balance_loss", _p(), *_swap(ok, i, ODD)) == -7
    assert _call("moe_balance_loss", _p(E=1025), *ok) == -2
    # logits, mask, counts, dloss, dlogits, stream
    ok = [F, None, F, F, F, None]
    for i in (0, 2, 3, 4):
        assert _call("moe_balance_loss_backward", _p(), *_swap(ok, i, None)) == -1
    for i in (0, 4):
        assert _call("moe_balance_loss_backward", _p(), *_swap(ok, i, ODD)) == -7


def test_router_backward():
    p = _p(T=1024)
    # dlogits, x, w_router, dx_in, dx, dw_router, ws, ws_bytes, stream
    ok = [F, F, F, None, ctypes.c_void_p(0x2000), F, F, BIG, None]
    for i in (0, 1, 2, 4, 5, 6):
        assert _call("moe_router_backward", p, *_swap(ok, i, None)) == -1
    for i in (0, 1, 2, 3, 4, 5, 6):
        assert _call("moe_router_backward", p, *_swap(ok, i, ODD)) == -7
    assert _call("moe_router_backward", p, *_swap(ok, 4, F)) == -7                     # dx is x
    assert _call("moe_router_backward", p, *_swap(ok, 7, 16)) == -4
    n = ctypes.c_size_t()
    assert _call("moe_router_backward_workspace_bytes", _p(T=1), ctypes.byref(n)) == 0 and n.value == 0


def test_forward_quantized():
    # x, xq, xq_scale, w_router, logits, packed, y, idx, gate, counts, offsets, pos, stats, ws, ws_bytes, stream
    ok = [None, F, F, None, F, F, F, None, None, None, None, None, None, F, BIG, None]
    name = "moe_forward_quantized"
    p = _p(act="mxfp8", logits_given=True)
    assert _call(name, _p(logits_given=True), *ok) == -3
    assert _call(name, _p(act="mxfp8", d=128, logits_given=True), *ok) == -2           # quantises per routed row
    for i in (1, 2, 4, 5, 6, 13):
        assert _call(name, p, *_swap(ok, i, None)) == -1
    assert _call(name, _p(act="mxfp8"), *_swap(ok, 3, F)) == -1                        # a learned router reads x
    assert _call(name, p, *_swap(ok, 1, ODD)) == -7
    assert _call(name, p, *_swap(ok, 2, ctypes.c_void_p(0x1002))) == -7
    assert _call(name, p, *_swap(ok, 14, 64)) == -4


def test_backward_aux():
    p = _p(act="mxfp8")
    n = ctypes.c_size_t()
    assert _call("moe_backward_aux_workspace_bytes", p, ctypes.byref(n)) == 0
    need, fws = n.value, B.workspace_bytes(p)
    assert need >= B.backward_workspace_bytes(p)
    given = _p(act="mxfp8", logits_given=True)
    assert _call("moe_backward_aux_workspace_bytes", given, ctypes.byref(n)) == 0
    assert n.value == B.backward_workspace_bytes(given)
    assert _call("moe_backward_aux_workspace_bytes", _p(identity=True), ctypes.byref(n)) == -3
    G = ctypes.c_void_p(0x3000)
    # dy, x, w_router, packed_w, packed_bwd, idx, gate, offsets, pos, fwd_ws, fwd_ws_bytes, dx, dlogits, dw_gate,
    # dw_up, dw_down, dw_router, ws, ws_bytes, stream, dlogits_aux, xq
    ok = [F, F, F, None, F, None, None, None, None, F, fws, F, F, F, F, F, F, F, need, None, G, F]
    name = "moe_backward_aux"
    assert _call(name, p, *_swap(ok, 0, None)) == -1
    assert _call(name, p, *_swap(ok, 18, need - 1)) == -4
    assert _call(name, p, *_swap(ok, 20, F)) == -7                                     # aux is dlogits
    for i in (1, 2, 11, 12, 17, 21):                                                   # x, w_router, dx, dlogits, ws, xq
        assert _call(name, p, *_swap(ok, i, ODD)) == -7
    assert _call(name, _p(), *ok) == -3                                                # codes of a bf16 block
    assert _call(name, _p(act="mxfp8", d=128), *ok) == -2


def test_decode():
    n = ctypes.c_size_t()
    for kw, st in [(dict(T=257), -2), (dict(d=192), -2), (dict(H=192), -2), (dict(act="f32"), -3),
                   (dict(identity=True), -3), (dict(T=256), 0), (dict(act="mxfp8"), 0),
                   # h [T k][2][H] bfloat16 reaches 2^32 bytes
                   (dict(T=256, E=16, k=16, d=128, H=1 << 18, act="mxfp8"), -2),
                   (dict(T=255, E=16, k=16, d=128, H=1 << 18, act="mxfp8"), 0)]:
        assert _call("moe_decode_workspace_bytes", _p(**kw), ctypes.byref(n)) == st
    p = _p(logits_given=True)
    assert B.decode_weight_bytes(p) == 8 * 3 * 256 * 256 * 17 // 32
    Y = ctypes.c_void_p(0x2000)
    # x, topk_idx, topk_gate, packed, y, ws, ws_bytes, stream
    ok = [F, F, F, F, Y, F, BIG, None]
    for i in range(6):
        assert _call("moe_decode_experts", p, *_swap(ok, i, None)) == -1
    for i in (0, 3, 4, 5):
        assert _call("moe_decode_experts", p, *_swap(ok, i, ODD)) == -7
    assert _call("moe_decode_experts", p, *_swap(ok, 4, F)) == -7                      # y is x
    assert _call("moe_decode_experts", p, *_swap(ok, 6, 64)) == -4
    # x, w_router, logits, packed, y, topk_idx, topk_gate, ws, ws_bytes, stream
    ok = [F, None, F, F, Y, None, None, F, BIG, None]
    for i in (0, 2, 3, 4, 7):
        assert _call("moe_decode", p, *_swap(ok, i, None)) == -1
    assert _call("moe_decode", _p(), *ok) == -1                                        # learned router without weights
    assert _call("moe_decode", p, *_swap(ok, 2, ODD)) == -7
    assert _call("moe_decode", p, *_swap(ok, 8, 64)) == -4
    # w_gate, w_up, w_down, packed, stream
    ok = [F, F, F, F, None]
    for i in range(4):
        assert _call("moe_pack_weights_decode", p, *_swap(ok, i, None)) == -1
    assert _call("moe_pack_weights_decode", p, *_swap(ok, 3, ODD)) == -7


def test_binding_checks_shapes_types_and_place():
    p = _p(T=4)
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    op = B.Norm(p, "cpu")
    with pytest.raises(ValueError, match="residual: expected"):
        op(x, w)
    with pytest.raises(ValueError, match="weight"):
        op(x, w.float(), residual=x)
    with pytest.raises(ValueError, match="device tensor"):
        op(x, w, residual=x)
    with pytest.raises(ValueError, match="residual: not expected"):
        B.Norm(p, "cpu", residual=False)(x, w, residual=x)
    with pytest.raises(ValueError, match="rstd"):
        B.NormBackward(p, "cpu")(x, x, w, torch.zeros(5))
    bal = B.BalanceLoss(p, "cpu")
    with pytest.raises(ValueError, match="mask"):
        bal(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), mask=torch.zeros(4, dtype=torch.bool))
    with pytest.raises(ValueError, match="idx"):
        bal(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64))
    with pytest.raises(ValueError, match="dloss"):
        bal.backward(torch.zeros(4, 8), torch.zeros(1))
    with pytest.raises(ValueError, match="w_router"):
        B.RouterBackward(p, "cpu")(torch.zeros(4, 8), x, torch.zeros(8, 256, dtype=torch.bfloat16))
    dec = B.Decode(p, "cpu")
    with pytest.raises(ValueError, match="packed"):
        dec.experts(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(8, dtype=torch.uint8))
    pm = _p(T=4, act="mxfp8", logits_given=True)
    with pytest.raises(ValueError, match="xq_scale"):
        B.Forward(pm, "cpu")(None, logits=torch.zeros(4, 8), xq=torch.zeros(4, 256, dtype=torch.uint8),
                             xq_scale=torch.zeros(4, 4, dtype=torch.uint8))


def test_operators_keep_their_problem_and_check_buffers_put_in_place():
    p = _p(T=4)
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    op = B.Norm(p, "cpu")
    p.T = 4096                                                # another problem: the operator's stays
    assert op.p.T == 4 and op.y.shape == (4, 256)
    with pytest.raises(ValueError, match="device tensor"):
        op(x, w, residual=x)
    p.T = 4
    for make, name in ((B.Norm, "y"), (B.Norm, "sum"), (B.NormBackward, "ds"), (B.BalanceLoss, "dlogits"),
                       (B.RouterBackward, "dx"), (B.Decode, "y"), (B.Decode, "idx")):
        op = make(p, "cpu")
        own = getattr(op, name)
        for wrong in (own[:2], own.double()):
            with pytest.raises(ValueError, match=name):
                setattr(op, name, wrong)
        with pytest.raises(ValueError, match="device tensor"):
            setattr(op, name, own.clone())
        assert getattr(op, name) is own
    op = B.Norm(p, "cpu", residual=False)
    assert op.sum is None
    with pytest.raises(ValueError, match="sum"):              # a buffer it was made without has a size too
        op.sum = x[:1]
    dec = B.Decode(p, "cpu")
    dec.idx = dec.gate = None
    assert dec.idx is None
