"""The operators around the block as they are used together (marked gpu): norm,
block, balance loss and all gradients of a training step against a float64
chain; an MXFP8 block fed with the norm's codes; norm and decode for serving;
each replayed from a graph.

Bars as the block's own backward tests (normwise: float32 1e-5, bf16 2e-2);
the float32 chain is held to the float64 one from its inputs on, the bf16
chains stage by stage on the stored values."""
import numpy as np
import pytest
import torch

from oracle import block_ops as Q
from oracle import moe_backward as BW
from oracle import moe_oracle as O
from routing_dispatch_grouped_router_amd import binding as B
from routing_dispatch_grouped_router_amd import workloads as W
from routing_dispatch_grouped_router_amd.workloads import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-6
DLOSS = (0.02, 0.003)
TOL = {"f32": 1e-5, "bf16": 2e-2, "mxfp8": 2e-2}


class Step:
    """A training step of a pre-norm block: everything preallocated, run() enqueues it."""

    def __init__(self, w: W.Workload, quantized: bool, padded: int = 0, keep: bool = False):
        self.w = w
        host = W.make_inputs(w)
        rng = np.random.default_rng(w.seed + 99)
        dt = B.storage_dtype(w.act)

        def draw(*shape, scale=1.0, mean=0.0):
            return torch.from_numpy((mean + scale * rng.standard_normal(shape)).astype(np.float32)).to(dt)
        self.host = dict(host, residual=draw(w.T, w.d), weight=draw(w.d, scale=0.1, mean=1.0), dy=draw(w.T, w.d),
                         dsum=draw(w.T, w.d))
        self.dev = {k: (None if v is None else v.to(DEV)) for k, v in self.host.items()}
        self.mask = None
        if padded:
            self.mask = torch.ones(w.T, dtype=torch.uint8, device=DEV)
            self.mask[-padded:] = 0
        self.dloss = torch.tensor(DLOSS, device=DEV)
        p = self.p = B.problem(w.T, w.d, w.E, w.k, w.H, w.act, logits_given=w.router != "learned",
                                 keep_gate_up=keep)
        d = self.dev
        self.packed = B.pack_weights(p, d["w_gate"], d["w_up"], d["w_down"])
        self.packed_bwd = B.pack_weights_backward(p, d["w_gate"], d["w_up"], d["w_down"])
        self.norm = B.Norm(p, DEV, eps=EPS, quantized=quantized)
        self.fwd = B.Forward(p, DEV)
        self.bal = B.BalanceLoss(p, DEV)
        self.bwd = B.Backward(p, DEV, aux=True)
        self.nbwd = B.NormBackward(p, DEV)
        if d["logits"] is not None:
            self.fwd.logits.copy_(d["logits"])

    def run(self):
        d, f = self.dev, self.fwd
        xn = self.norm(d["x"], d["weight"], residual=d["residual"])
        lg = f.logits if d["logits"] is not None else None
        f(xn, packed=self.packed, w_router=d["w_router"], logits=lg, xq=self.norm.q, xq_scale=self.norm.q_scale)
        self.bal(f.logits, f.idx, mask=self.mask)
        aux = self.bal.backward(f.logits, self.dloss, mask=self.mask)
        g = self.bwd(f, d["dy"], self.packed, self.packed_bwd, x=xn, w_router=d["w_router"], dlogits_aux=aux,
                     xq=self.norm.q)
        n = self.nbwd(g["dx"], self.norm.sum, d["weight"], self.norm.rstd, dsum=d["dsum"])
        return dict(g, **n, y=f.y, sum=self.norm.sum, loss=self.bal.loss, counts=self.bal.counts)


def _close(name, got, ref, tol):
    got = as_f64(got)
    scale = np.max(np.abs(ref))
    err = np.max(np.abs(got - ref))
    assert err <= tol * scale, f"{name}: normwise {err / max(scale, 1e-300):.3e} > {tol}"


CASES = [
    (W.Workload("chain_f32_learned", T=333, d=192, E=12, k=3, H=128, act="f32", router="learned", seed=5101), False, 0),
    (W.Workload("chain_bf16_learned", T=600, d=256, E=8, k=4, H=192, act="bf16", router="learned", seed=5102), False, 50),
    (W.Workload("chain_bf16_e20", T=301, d=64, E=20, k=2, H=64, act="bf16", router="learned", seed=5103), False, 0),
    (W.Workload("chain_bf16_random", T=500, d=384, E=32, k=4, H=128, act="bf16", router="random", seed=5104), False, 0),
    (W.Workload("chain_mx_learned", T=400, d=256, E=8, k=2, H=128, act="mxfp8", router="learned", seed=5105), True, 7),
    (W.Workload("chain_mx_random", T=300, d=384, E=16, k=4, H=256, act="mxfp8", router="random", seed=5106), True, 0),
    (W.Workload("chain_mx_d128", T=200, d=128, E=8, k=2, H=128, act="mxfp8", router="learned", seed=5107), False, 0),
]


@pytest.mark.parametrize("w, quantized, padded", CASES, ids=[c[0].name for c in CASES])
def test_training_step(w, quantized, padded):
    print(f"[chain] {w.describe()}", flush=True)
    st = Step(w, quantized, padded)
    out = {k: (None if v is None else v.clone()) for k, v in st.run().items()}
    torch.cuda.synchronize()
    h, tol = st.host, TOL[w.act]
    exact = w.act == "f32"
    x, r, wn, dy, dsum = (as_f64(h[n]) for n in ("x", "residual", "weight", "dy", "dsum"))
    s, rstd, y = Q.rmsnorm(x, r, wn, EPS)
    if exact:
        xn, logits = y, as_f64(st.fwd.logits)
        _close("logits", st.fwd.logits, O.router_logits(y, as_f64(h["w_router"])), tol)
    else:
        _close("xn", st.norm.y, y, tol)
        xn, logits, s = as_f64(st.norm.y), as_f64(st.fwd.logits), as_f64(st.norm.sum)
    wg, wu, wd = (as_f64(h[n]) for n in ("w_gate", "w_up", "w_down"))
    fo = O.forward(xn, w.E, w.k, w.act, wg, wu, wd, logits=logits)
    assert np.array_equal(fo["idx"], st.fwd.idx.cpu().numpy())
    _close("y", out["y"], fo["y"], tol)
    mask = None if st.mask is None else st.mask.cpu().numpy()
    loss, counts, _ = Q.balance_loss(logits, fo["idx"], mask)
    _close("loss", out["loss"], loss, 400 * 2.0 ** -24)
    assert np.array_equal(out["counts"].cpu().numpy(), counts)
    aux = Q.balance_loss_backward(logits, counts, w.k, DLOSS, mask)
    if w.act == "mxfp8":
        q = [O.expert_weights(wg, wu, wd, e, "mxfp8") for e in range(w.E)]
        wg, wu, wd = (np.stack([t[i] for t in q]) for i in range(3))
    ref = BW.backward(xn, dy, fo, w.act, wg, wu, wd)         # the block without its router's product
    dl = ref["dlogits"] + aux
    _close("dlogits", out["dlogits"], dl, tol)
    dx = ref["dx"]
    if w.router == "learned":
        wr = as_f64(h["w_router"])
        dx = dx + dl @ wr.T
        _close("dw_router", out["dw_router"], xn.T @ dl, tol)
    _close("dx", out["dx"], dx, tol)
    for name in ("dw_gate", "dw_up", "dw_down"):
        _close(name, out[name], ref[name], tol)
    ds, dweight = Q.rmsnorm_backward(dx, dsum, s, wn, eps=EPS)
    _close("ds", out["ds"], ds, tol)
    _close("dweight", out["dweight"], dweight, tol)


@pytest.mark.parametrize("keep", [False, True], ids=["recompute", "keep_gate_up"])
@pytest.mark.parametrize("w", [c[0] for c in CASES if c[1]], ids=[c[0].name for c in CASES if c[1]])
def test_quantised_rows_give_the_same_block(w, keep):
    """moe_forward_quantized and its backward, bit for bit those of the bf16 rows."""
    st = Step(w, True, keep=keep)
    out = {k: (None if v is None else v.clone()) for k, v in st.run().items()}
    idx, pos = st.fwd.idx.clone(), st.fwd.pos.clone()
    st.norm.q = st.norm.q_scale = None
    st.fwd.ws.fill_(255)
    for k, v in st.run().items():
        assert v is None or torch.equal(v, out[k]), k
    assert torch.equal(idx, st.fwd.idx) and torch.equal(pos, st.fwd.pos)
    # given logits need no bf16 rows at all
    if w.router != "learned":
        st2 = Step(w, True)
        st2.norm.y = None
        st2.norm(st2.dev["x"], st2.dev["weight"], residual=st2.dev["residual"])
        y = st2.fwd(None, packed=st2.packed, logits=st2.fwd.logits, xq=st2.norm.q, xq_scale=st2.norm.q_scale)
        assert torch.equal(y, out["y"])


def test_aux_of_zeros_is_the_sparse_backward():
    """With nothing to add the dense router gradients are the sparse ones up to their rounding."""
    w = CASES[1][0]
    st = Step(w, False)
    st.dloss.zero_()
    dense = {k: (None if v is None else v.clone()) for k, v in st.run().items()}
    sparse = st.bwd(st.fwd, st.dev["dy"], st.packed, st.packed_bwd, x=st.norm.y, w_router=st.dev["w_router"])
    for k in ("dlogits", "dw_gate", "dw_up", "dw_down"):
        assert torch.equal(dense[k], sparse[k]), k
    for k, tol in (("dx", 2.0 ** -7), ("dw_router", 1e-5)):    # one bf16 step; float32 sums in another order
        _close(k, dense[k], as_f64(sparse[k]), tol)


def test_two_steps_at_once():
    """Two steps with buffers of their own on two streams, neither waiting for the other."""
    steps = [Step(*CASES[4]), Step(*CASES[1])]
    want = []
    for st in steps:
        st.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in _outputs(st)])
    for st in steps:
        for t in _outputs(st):
            t.fill_(3)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for st, s in zip(steps, streams):
            with torch.cuda.stream(s):
                st.run()
    torch.cuda.synchronize()
    for st, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(_outputs(st), w))


def _graph_replays(run, outputs, n=4):
    """run() captured, replayed with eager work between, each replay bit for bit the eager result."""
    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in outputs()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for i in range(n):
        for t in outputs():
            t.fill_(3)
        scratch = torch.randn(4096, device=DEV) * i
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outputs()):
            assert torch.equal(a, b), f"replay {i}"
        del scratch
        if i == 1:
            run()                                              # an eager pass between replays


@pytest.mark.parametrize("case", [1, 4, 5], ids=[CASES[i][0].name for i in (1, 4, 5)])
def test_training_step_in_a_graph(case):
    st = Step(*CASES[case])
    _graph_replays(st.run, lambda: _outputs(st))


def _outputs(st):
    b, n = st.bwd, st.nbwd
    return [t for t in (st.fwd.y, st.norm.sum, st.bal.loss, st.bal.counts_live, b.dx, b.dlogits, b.dw_gate, b.dw_up,
                        b.dw_down, b.dw_router, n.ds, n.dweight) if t is not None]


@pytest.mark.parametrize("T", [1, 20])
def test_serving_step(T):
    """norm, then the 4-bit block, for one token and a few; on another stream and from a graph too."""
    d, E, k, H = 512, 16, 4, 256
    rng = np.random.default_rng(T)

    def draw(*shape, scale=1.0, mean=0.0):
        return torch.from_numpy((mean + scale * rng.standard_normal(shape)).astype(np.float32)).to(torch.bfloat16)
    x, r, wn, wr = draw(T, d), draw(T, d), draw(d, scale=0.1, mean=1.0), draw(d, E, scale=0.05)
    ws = [draw(E, d, H, scale=0.05), draw(E, d, H, scale=0.05), draw(E, H, d, scale=0.05)]
    p = B.problem(T, d, E, k, H, "bf16")
    packed = B.pack_weights_decode(p, *(t.to(DEV) for t in ws))
    norm, dec = B.Norm(p, DEV, eps=EPS), B.Decode(p, DEV)
    xd, rd, wnd, wrd = (t.to(DEV) for t in (x, r, wn, wr))

    def run(stream=None):
        return dec(norm(xd, wnd, residual=rd, stream=stream), packed, w_router=wrd, stream=stream)
    y = run().clone()
    _, _, yn = Q.rmsnorm(as_f64(x), as_f64(r), as_f64(wn), EPS)
    _close("xn", norm.y, yn, 2.0 ** -8)
    ref, err = Q.decode_experts(as_f64(norm.y), dec.idx.cpu().numpy(), as_f64(dec.gate),
                                *Q.decode_weights(packed.cpu().numpy(), E, d, H))
    assert np.all(np.abs(as_f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * err)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dec.y.fill_(0)
    s.wait_stream(torch.cuda.current_stream())
    run(stream=s)
    s.synchronize()
    assert torch.equal(dec.y, y)
    _graph_replays(run, lambda: [dec.y, dec.idx, norm.sum])
