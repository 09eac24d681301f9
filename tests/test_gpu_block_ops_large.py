"""The operators around the block on tensors past 2^31 elements or 2^32 bytes
(marked gpu): what they compute for the last rows or experts is bit for bit
what they compute for these alone, which the small tests hold to the oracle.
The row operators as MXFP8 problems: the others' token rows are refused from
2^32 bytes on."""
import pytest
import torch

from routing_dispatch_grouped_router_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _rand(shape, dtype=torch.bfloat16):
    return torch.randn(shape, dtype=dtype, device=DEV)


def test_norm_rows():
    T, d, n = 262200, 8320, 3                                 # 2.18e9 values a tensor
    print(f"[large norm] T={T} d={d}", flush=True)
    x, r, w = _rand((T, d)), _rand((T, d)), _rand((d,))
    op = B.Norm(B.problem(T, d, 1, 1, 128, "mxfp8"), DEV)
    op.y, op.sum = x, r                                       # in place, as far as the memory goes too
    last = [t[-n:].clone() for t in (x, r)]
    op(x, w, residual=r)
    few = B.Norm(B.problem(n, d, 1, 1, 128, "mxfp8"), DEV)
    few(last[0], w, residual=last[1])
    assert torch.equal(op.y[-n:], few.y) and torch.equal(op.sum[-n:], few.sum) and torch.equal(op.rstd[-n:], few.rstd)
    assert torch.equal(op.q[-n:], few.q) and torch.equal(op.q_scale[-n:], few.q_scale)
    dy = x
    bwd = B.NormBackward(B.problem(T, d, 1, 1, 128, "mxfp8"), DEV)
    g = bwd(dy, r, w, op.rstd)
    want = B.NormBackward(B.problem(n, d, 1, 1, 128, "mxfp8"), DEV)(dy[-n:], r[-n:], w, op.rstd[-n:])
    assert torch.equal(g["ds"][-n:], want["ds"])
    assert g["dweight"].isfinite().all()


@pytest.mark.parametrize("E", [8, 72])
def test_router_gradient_rows(E):
    T, d, n = 262200, 8320, 70
    print(f"[large router gradients] T={T} d={d} E={E}", flush=True)
    x, w, dl = _rand((T, d)), _rand((d, E)), _rand((T, E), torch.float32)
    last = x[-n:].clone()
    op = B.RouterBackward(B.problem(T, d, E, 1, 128, "mxfp8"), DEV)
    g = op(dl, x, w, dx_in=x)
    few = B.RouterBackward(B.problem(n, d, E, 1, 128, "mxfp8"), DEV)
    want = few(dl[-n:].contiguous(), last, w, dx_in=last)
    assert torch.equal(g["dx"][-n:], want["dx"])
    # the weight gradient, from the last token alone
    dl[:-1] = 0
    g = op(dl, x, w)
    want = x[-1].float()[:, None] * dl[-1][None, :]
    assert torch.allclose(g["dw_router"], want, rtol=2.0 ** -20, atol=0)


def test_decode_weights():
    T, d, E, k, H = 40, 4096, 352, 2, 2048                    # 4.7 GB of packed weights
    print(f"[large decode] T={T} d={d} E={E} H={H}", flush=True)
    p = B.problem(T, d, E, k, H, "bf16")
    n = B.decode_weight_bytes(p)
    assert n > 2 ** 32
    packed = torch.empty(n, dtype=torch.uint8, device=DEV)
    codes = E * 3 * d * H // 2
    packed[:codes].random_(0, 256)
    packed[codes:].random_(118, 122)                          # scales 2^-9 .. 2^-6
    x = _rand((T, d))
    gate = torch.rand((T, k), device=DEV)
    idx = torch.randint(0, 2, (T, k), dtype=torch.int32, device=DEV)
    y = B.Decode(p, DEV).experts(x, idx + (E - 2), gate, packed)
    # the last two experts as a block of two
    p2 = B.problem(T, d, 2, k, H, "bf16")
    two, off = [], 0
    for per in (H * d, d * H // 2, H * d // 16, d * H // 32):
        two.append(packed[off + (E - 2) * per:off + E * per])
        off += E * per
    assert off == n
    y2 = B.Decode(p2, DEV).experts(x, idx, gate, torch.cat(two))
    assert y.isfinite().all() and y.any() and torch.equal(y, y2)


def test_replayed_from_a_graph():
    """The kernels that only many experts or tokens reach, captured once and replayed on other inputs with eager calls
    of the same operators between."""
    T, d, E, k, H = 64, 1024, 80, 2, 512
    p = B.problem(T, d, E, k, H, "bf16")
    w = [0.05 * _rand(s) for s in ((E, d, H), (E, d, H), (E, H, d))]
    packed = B.pack_weights_decode(p, *w)
    x, gate = _rand((T, d)), torch.rand((T, k), device=DEV)
    idx = torch.randint(0, E, (T, k), dtype=torch.int32, device=DEV)
    dec = B.Decode(p, DEV)
    Tr, dr, Er = 70001, 64, 24
    pr = B.problem(Tr, dr, Er, 1, 64, "bf16")
    dl, xr, wr, add = _rand((Tr, Er), torch.float32), _rand((Tr, dr)), _rand((dr, Er)), _rand((Tr, dr))
    rb = B.RouterBackward(pr, DEV)
    pb = B.problem(300, 64, 16, 2, 64, "f32")
    logits, choice = _rand((300, 16), torch.float32), torch.randint(0, 16, (300, 2), dtype=torch.int32, device=DEV)
    bal = B.BalanceLoss(pb, DEV)

    def run(dec, rb, bal):
        dec.experts(x, idx, gate, packed)
        rb(dl, xr, wr, dx_in=add)
        bal(logits, choice)
        return [dec.y, rb.dx, rb.dw_router, bal.loss, bal.counts_live]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(dec, rb, bal)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(dec, rb, bal)
    other = B.Decode(p, DEV), B.RouterBackward(pr, DEV), B.BalanceLoss(pb, DEV)
    for i in range(4):
        for t in (x, gate, dl, xr, add, logits):
            t.mul_(0.75).add_(0.125)
        idx.add_(7 * i).remainder_(E)
        want = [t.clone() for t in run(*other)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
