"""Layer norm, block, balance loss, all gradients, their norm and the AdamW step of
a block's weights, as a training program runs them, and the block for a few
tokens on the weights that the steps leave (marked gpu).

Bars as the block's own tests (normwise: float32 1e-5, bf16 2e-2): the float32
chain is held to the float64 one from its inputs to the gradients, the step to
the formula from the gradients it was given (tests/test_gpu_adamw.py holds it
to its roundings)."""
import numpy as np
import pytest
import torch

from oracle import block_ops as R
from oracle import moe_backward as BW
from oracle import moe_oracle as O
from oracle import training_ops as Q
from routing_dispatch_grouped_router_amd import binding as B
from routing_dispatch_grouped_router_amd import workloads as W
from routing_dispatch_grouped_router_amd.workloads import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS, DLOSS, BETAS, LR, DECAY, MAX_NORM = 1e-5, (0.02, 0.003), (0.9, 0.95), 1e-3, 0.1, 0.5
TOL = {"f32": 1e-5, "bf16": 2e-2, "mxfp8": 2e-2}
NAMES = ("w_gate", "w_up", "w_down", "w_router", "weight", "bias")


class Train:
    """A pre-norm block's training step: everything preallocated, run() enqueues it."""

    def __init__(self, w: W.Workload, states: str, padded: int = 0):
        self.w = w
        host = W.make_inputs(w)
        rng = np.random.default_rng(w.seed + 7)
        dt = B.storage_dtype(w.act)

        def draw(*shape, scale=1.0, mean=0.0):
            return torch.from_numpy((mean + scale * rng.standard_normal(shape)).astype(np.float32)).to(dt)
        self.host = dict(host, residual=draw(w.T, w.d), weight=draw(w.d, scale=0.1, mean=1.0), bias=draw(w.d, scale=0.1),
                         dy=draw(w.T, w.d), dsum=draw(w.T, w.d))
        self.dev = d = {k: (None if v is None else v.to(DEV)) for k, v in self.host.items()}
        self.mask = None
        if padded:
            self.mask = torch.ones(w.T, dtype=torch.uint8, device=DEV)
            self.mask[-padded:] = 0
        self.dloss = torch.tensor(DLOSS, device=DEV)
        p = self.p = B.problem(w.T, w.d, w.E, w.k, w.H, w.act)
        self.norm, self.fwd, self.bal = B.LayerNorm(p, DEV, eps=EPS), B.Forward(p, DEV), B.BalanceLoss(p, DEV)
        self.bwd, self.nbwd = B.Backward(p, DEV, aux=True), B.LayerNormBackward(p, DEV)
        grads = [self.bwd.dw_gate, self.bwd.dw_up, self.bwd.dw_down, self.bwd.dw_router, self.nbwd.dweight, self.nbwd.dbias]
        self.opt = B.AdamW([d[n] for n in NAMES], grads, lr=LR, betas=BETAS, eps=1e-8, weight_decay=[DECAY] * 4 + [0.0] * 2,
                           master=True if w.act != "f32" and states == "f32" else None, states=states, seed=3)

    def gradients(self):
        d, f = self.dev, self.fwd
        self.packed = B.pack_weights(self.p, d["w_gate"], d["w_up"], d["w_down"])
        packed_bwd = B.pack_weights_backward(self.p, d["w_gate"], d["w_up"], d["w_down"])
        xn = self.norm(d["x"], d["weight"], d["bias"], residual=d["residual"])
        f(xn, packed=self.packed, w_router=d["w_router"], xq=self.norm.q, xq_scale=self.norm.q_scale)
        self.bal(f.logits, f.idx, mask=self.mask)
        aux = self.bal.backward(f.logits, self.dloss, mask=self.mask)
        g = self.bwd(f, d["dy"], self.packed, packed_bwd, x=xn, w_router=d["w_router"], dlogits_aux=aux, xq=self.norm.q)
        n = self.nbwd(g["dx"], self.norm.sum, d["weight"], self.norm.mean, self.norm.rstd, dsum=d["dsum"])
        return dict(g, **n)

    def run(self):
        self.gradients()
        self.opt(clip=self.opt.grad_norm(MAX_NORM))

    def state(self):
        o = self.opt
        lists = [o.weights, o.m, *([o.v] if o.v else [o.r, o.m_scale, o.r_scale]), [m for m in o.master or [] if m is not None]]
        return [t for ts in lists for t in ts] + [o.step, o.norm, self.nbwd.ds]


def _close(name, got, ref, tol):
    got, scale = as_f64(got), np.max(np.abs(ref))
    err = np.max(np.abs(got - ref))
    assert err <= tol * scale, f"{name}: normwise {err / max(scale, 1e-300):.3e} > {tol}"


CASES = [
    (W.Workload("train_f32", T=333, d=192, E=12, k=3, H=128, act="f32", router="learned", seed=6101), "f32", 0),
    (W.Workload("train_f32_8bit", T=100, d=128, E=8, k=2, H=64, act="f32", router="learned", seed=6102), "8bit", 9),
    (W.Workload("train_bf16_master", T=600, d=256, E=8, k=4, H=192, act="bf16", router="learned", seed=6103), "f32", 50),
    (W.Workload("train_bf16_8bit", T=301, d=64, E=20, k=2, H=64, act="bf16", router="learned", seed=6104), "8bit", 0),
    (W.Workload("train_mx_8bit", T=400, d=256, E=8, k=2, H=128, act="mxfp8", router="learned", seed=6105), "8bit", 7),
]
IDS = [c[0].name for c in CASES]


@pytest.mark.parametrize("w, states, padded", CASES, ids=IDS)
def test_training_step(w, states, padded):
    print(f"[train] {w.describe()} {states}", flush=True)
    st = Train(w, states, padded)
    h, tol = st.host, TOL[w.act]
    out = {k: (None if v is None else v.clone()) for k, v in st.gradients().items()}
    torch.cuda.synchronize()
    x, r, wn, bn, dy, dsum = (as_f64(h[n]) for n in ("x", "residual", "weight", "bias", "dy", "dsum"))
    s, mean, rstd, xn = Q.layer_norm(x, r, wn, bn, EPS)
    if w.act != "f32":                                       # the rest from the stored values, stage by stage
        _close("xn", st.norm.y, xn, tol)
        xn, s, mean, rstd = (as_f64(t) for t in (st.norm.y, st.norm.sum, st.norm.mean, st.norm.rstd))
    logits = as_f64(st.fwd.logits)
    wg, wu, wd, wr = (as_f64(h[n]) for n in ("w_gate", "w_up", "w_down", "w_router"))
    fo = O.forward(xn, w.E, w.k, w.act, wg, wu, wd, logits=logits)
    assert np.array_equal(fo["idx"], st.fwd.idx.cpu().numpy())
    mask = None if st.mask is None else st.mask.cpu().numpy()
    _, counts, _ = R.balance_loss(logits, fo["idx"], mask)
    if w.act == "mxfp8":
        q = [O.expert_weights(wg, wu, wd, e, "mxfp8") for e in range(w.E)]
        wg, wu, wd = (np.stack([t[i] for t in q]) for i in range(3))
    ref = BW.backward(xn, dy, fo, w.act, wg, wu, wd)
    dl = ref["dlogits"] + R.balance_loss_backward(logits, counts, w.k, DLOSS, mask)
    ds, dweight, dbias = Q.layer_norm_backward(ref["dx"] + dl @ wr.T, dsum, s, wn, mean, rstd)
    want = dict(dw_gate=ref["dw_gate"], dw_up=ref["dw_up"], dw_down=ref["dw_down"], dw_router=xn.T @ dl, ds=ds,
                dweight=dweight, dbias=dbias)
    for name, v in want.items():
        _close(name, out[name], v, tol)
    # the step from those gradients
    before = [t.clone() for t in st.opt.weights]
    norm = st.opt.grad_norm(MAX_NORM)
    st.opt(clip=norm)
    torch.cuda.synchronize()
    n, factor = Q.grad_norm([as_f64(g) for g in st.opt.grads], MAX_NORM)
    assert abs(float(norm[0]) - n) <= 1e-6 * n and abs(float(norm[1]) - factor) <= 1e-6 * factor and factor < 1
    for i, name in enumerate(NAMES):
        w0, g = as_f64(before[i]), as_f64(st.opt.grads[i]) * factor
        w1, _, _ = Q.adamw(w0, g, 0, 0, 1, LR, BETAS, 1e-8, DECAY if i < 4 else 0.0)
        got = as_f64(st.opt.weights[i])
        step = 2.0 ** -23 if w.act == "f32" else 2.0 ** -7   # of the weight's type; to nearest half of that
        assert np.all(np.abs(got - w1) <= step * np.abs(w1) + 1e-5 * LR), name
        if st.opt.master is not None:   # a weight near 1 stays: the step, LR, is less than half of its bf16 step
            _close(name, st.opt.master[i], w1, 1e-6)
            got = as_f64(st.opt.master[i])
        assert np.any(got != w0)
    assert st.opt.step.tolist() == [1, 0]


@pytest.mark.parametrize("case", range(len(CASES)), ids=IDS)
def test_steps_in_a_graph(case):
    """Whole steps captured and replayed, with eager work between: bit for bit the eager steps, weights and states too."""
    eager, graphed = Train(*CASES[case]), Train(*CASES[case])
    eager.run()
    graphed.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        graphed.run()
    for i in range(4):
        x = torch.randn(eager.w.T, eager.w.d, device=DEV)
        for t in (eager, graphed):
            t.dev["x"].copy_(x)
        eager.run()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.state(), graphed.state()):
            assert torch.equal(a, b), f"replay {i}"
    assert eager.opt.step.tolist() == [5, 0]


@pytest.mark.parametrize("case", [0, 2, 4], ids=[IDS[i] for i in (0, 2, 4)])
@pytest.mark.parametrize("T", [1, 6])
def test_trained_weights_for_a_few_tokens(case, T):
    """Norm and the block for a few tokens on the weights after two steps: the rows that the block gives, eager and replayed."""
    st = Train(*CASES[case])
    for _ in range(2):
        st.run()
    w, d, tol = st.w, st.dev, TOL[st.w.act]
    st.packed = B.pack_weights(st.p, d["w_gate"], d["w_up"], d["w_down"])
    p = B.problem(T, w.d, w.E, w.k, w.H, w.act)
    norm, few = B.LayerNorm(p, DEV, eps=EPS, quantized=False), B.ForwardFew(p, DEV)
    x, r = d["x"][:T].contiguous(), d["residual"][:T].contiguous()

    def run():
        return few(norm(x, d["weight"], d["bias"], residual=r), st.packed, w_router=d["w_router"])
    y = run().clone()
    xn = as_f64(norm.y)
    logits = xn @ as_f64(d["w_router"])
    wg, wu, wd = (as_f64(d[n]) for n in ("w_gate", "w_up", "w_down"))
    if w.act == "mxfp8":
        q = [O.expert_weights(wg, wu, wd, e, "mxfp8") for e in range(w.E)]
        wg, wu, wd = (np.stack([t[i] for t in q]) for i in range(3))
    _close("logits", few.logits, logits, 1e-5)
    ref, _ = R.decode_experts(xn, few.idx.cpu().numpy(), as_f64(few.gate), wg, wu, wd)
    _close("y", y, ref, tol)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(3):
        few.y.fill_(3)
        torch.randn(4096, device=DEV)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(few.y, y)
