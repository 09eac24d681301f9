"""The block for a few tokens on packed weights (moe_forward_few) against the float64 oracle (marked gpu).

Tolerances, from the arithmetic (u = 2^-24, half a float32 step): a sum of n
products in float32 is off by at most n u times the sum of their magnitudes;
what that makes of h and y is block_ops.decode_experts' bound, with h held to
2^-16 of it (two bfloat16 terms) or, for float32 blocks, to a rounding; y takes
half a step of its type.  A gate is a quotient of up to 16 exponentials of
float32 differences: 64 u of it."""
import numpy as np
import pytest
import torch

from oracle import block_ops as Q
from oracle import moe_oracle as O
from routing_dispatch_grouped_router_amd import binding as B
from routing_dispatch_grouped_router_amd.workloads import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "mxfp8": 2.0 ** -8}


def _rand(rng, shape, act, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(B.storage_dtype(act))


class Case:
    def __init__(self, T, d, E, k, H, act, seed=0, given=False, scale=0.05):
        rng = np.random.default_rng(seed + T * 31 + d + E)
        self.p = B.problem(T, d, E, k, H, act, logits_given=given)
        self.act = act
        self.x, self.w_router = _rand(rng, (T, d), act), _rand(rng, (d, E), act, 0.05)
        self.logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)) if given else None
        self.w = [_rand(rng, (E, d, H), act, scale), _rand(rng, (E, d, H), act, scale), _rand(rng, (E, H, d), act, scale)]
        self.dev = dict(x=self.x.to(DEV), w_router=None if given else self.w_router.to(DEV),
                        logits=self.logits.to(DEV) if given else None)
        self.packed = B.pack_weights(self.p, *(w.to(DEV) for w in self.w))
        self.op = B.ForwardFew(self.p, DEV)

    def run(self, op=None, mask=None, x=None, stream=None):
        op = self.op if op is None else op
        return op(self.dev["x"] if x is None else x, self.packed, w_router=self.dev["w_router"],
                  logits=self.dev["logits"], mask=mask, stream=stream)

    def values(self):
        """Weights as the kernels have them."""
        w = [as_f64(t) for t in self.w]
        if self.act != "mxfp8":
            return w
        q = [O.expert_weights(*w, e, "mxfp8") for e in range(self.p.n_experts)]
        return [np.stack([t[i] for t in q]) for i in range(3)]

    def check(self, mask=None):
        torch.cuda.synchronize()
        p, op = self.p, self.op
        x = as_f64(self.x)
        live = np.ones(p.T, bool) if mask is None else mask.cpu().numpy() != 0
        if self.logits is None:
            logits, wr = as_f64(op.logits), as_f64(self.w_router)
            bound = p.d_model * U * (np.abs(x) @ np.abs(wr)) + 1e-30
            assert np.all(np.abs(logits - x @ wr)[live] <= bound[live]), "logits"
        else:
            logits = as_f64(self.logits)
        order = np.argsort(-logits, axis=1, kind="stable")[:, :p.top_k]
        idx, gate = op.idx.cpu().numpy(), as_f64(op.gate)
        assert np.array_equal(idx[live], order[live]) and np.all(idx[~live] == -1) and np.all(gate[~live] == 0)
        z = np.exp(np.take_along_axis(logits, order, 1) - logits.max(axis=1, keepdims=True))
        z /= z.sum(axis=1, keepdims=True)
        assert np.all(np.abs(gate - z)[live] <= 64 * U * z[live]), "gates"
        ref, err = Q.decode_experts(np.where(live[:, None], x, 0), idx, gate, *self.values(),
                                    u_h=U if self.act == "f32" else 2.0 ** -16)
        got = as_f64(op.y)
        off = np.abs(got - ref) - (HALF[self.act] * np.abs(ref) + 1.01 * err)
        assert np.all(off <= 0), f"y: worst {off.max():.3e}"
        assert np.all(got[~live] == 0)


def _width(n, act):
    return -(-n // 128) * 128 if act == "mxfp8" else n


SHAPES = [(1, 64, 4, 4, 64), (1, 512, 64, 8, 256), (1, 2048, 8, 2, 1024), (2, 64, 1024, 16, 64), (3, 192, 12, 3, 128),
          (5, 1088, 20, 2, 448), (7, 256, 128, 4, 128), (9, 1024, 64, 8, 512), (13, 128, 99, 5, 192),
          (16, 320, 8, 4, 192), (17, 384, 8, 1, 320), (32, 128, 8, 2, 64), (32, 64, 1, 1, 64), (32, 128, 16, 16, 128),
          (31, 576, 32, 8, 64), (4, 4096, 16, 2, 128), (3, 128, 512, 4, 64), (2, 8448, 8, 2, 64),
          (21, 192, 8, 4, 192), (16, 128, 16, 8, 576)]


@pytest.mark.parametrize("act", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("T, d, E, k, H", SHAPES)
def test_forward_few(T, d, E, k, H, act):
    d, H = _width(d, act), _width(H, act)
    print(f"[few] T={T} d={d} E={E} k={k} H={H} {act}", flush=True)
    c = Case(T, d, E, k, H, act)
    for t in (c.op.y, c.op.logits, c.op.idx, c.op.gate):
        t.fill_(7)
    c.op.ws.fill_(255)
    c.run()
    c.check()
    first = [t.clone() for t in (c.op.y, c.op.logits, c.op.idx, c.op.gate)]
    c.run()
    assert all(torch.equal(a, b) for a, b in zip(first, (c.op.y, c.op.logits, c.op.idx, c.op.gate)))


@pytest.mark.parametrize("act", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("T, E, k", [(1, 8, 2), (6, 30, 7), (32, 4, 4)])
def test_given_logits(T, E, k, act):
    c = Case(T, 256, E, k, 128, act, given=True)
    before = c.dev["logits"].clone()
    c.run()
    c.check()
    assert torch.equal(before, c.dev["logits"])


def test_ties_go_to_the_lower_expert():
    c = Case(8, 128, 33, 6, 64, "bf16", given=True)
    rng = np.random.default_rng(3)
    c.logits = torch.from_numpy(rng.integers(-1, 2, (8, 33)).astype(np.float32))
    c.logits[0] = 0
    c.logits[1, ::2] = -0.0                                     # as 0
    c.logits[1, 1::2] = 0
    c.dev["logits"] = c.logits.to(DEV)
    c.run()
    c.check()
    assert c.op.idx[0].tolist() == c.op.idx[1].tolist() == list(range(6))


@pytest.mark.parametrize("act", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("given", [False, True])
def test_padded_tokens(act, given):
    """Rows that are padding hold NaN and do not matter; all padding is all zero."""
    c = Case(9, 256, 16, 3, 128, act, given=given)
    mask = torch.tensor([1, 0, 1, 1, 0, 1, 1, 0, 0], dtype=torch.uint8, device=DEV)
    c.run()
    want = [t.clone() for t in (c.op.y, c.op.idx, c.op.gate)]
    x = c.dev["x"].clone()
    x[mask == 0] = float("nan")
    if given:
        c.dev["logits"][mask == 0] = float("nan")
    c.run(mask=mask, x=x)
    c.check(mask)
    for a, b in zip(want, (c.op.y, c.op.idx, c.op.gate)):
        assert torch.equal(a[mask != 0], b[mask != 0])
    mask.zero_()
    c.run(mask=mask, x=x)
    assert not c.op.y.any() and (c.op.idx == -1).all() and not c.op.gate.any()


@pytest.mark.parametrize("act", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("T, d, E, k, H", [(32, 512, 8, 4, 256), (20, 384, 64, 6, 128), (9, 320, 12, 2, 64), (21, 256, 8, 4, 1088)])
def test_a_token_does_not_depend_on_its_batch(T, d, E, k, H, act):
    """Bit for bit the token alone, in a few, and in another order."""
    d, H = _width(d, act), _width(H, act)
    c = Case(T, d, E, k, H, act)
    want = c.run().clone()
    for n in (1, 2, 5, 8, 16):
        op = B.ForwardFew(B.problem(n, d, E, k, H, act), DEV)
        for t0 in range(0, T - n + 1, n):
            y = c.run(op, x=c.dev["x"][t0:t0 + n].contiguous())
            assert torch.equal(y, want[t0:t0 + n]), (n, t0)
    perm = torch.randperm(T, device=DEV)
    assert torch.equal(c.run(x=c.dev["x"][perm].contiguous()), want[perm])


@pytest.mark.parametrize("act", ["bf16", "mxfp8"])
def test_hidden_units_past_bfloat16(act):
    """A unit between bfloat16's and float32's largest values, 1.99988 2^127: h is the float32 product.  Infinite rows
    leave the others."""
    c = Case(2, 128, 4, 2, 128, act, given=True)
    c.x.zero_()
    c.x[0, 0], c.x[0, 1], c.x[1, 5] = 1.0078125 * 2.0 ** 40, 1.984375 * 2.0 ** 40, 1.0
    for w in c.w[:2]:
        w.zero_()
    c.w[0][:, 0, 3], c.w[1][:, 1, 3] = 2.0 ** 23, 2.0 ** 24
    c.w[2].mul_(2.0 ** -60)
    c.dev["x"].copy_(c.x)
    c.packed.copy_(B.pack_weights(c.p, *(w.to(DEV) for w in c.w)))
    c.run()
    c.check()
    assert c.op.y[0].any() and c.op.y.isfinite().all()
    want, x = c.op.y.clone(), c.dev["x"].clone()
    x[1] = float("inf")
    y = c.run(x=x)
    assert torch.equal(y[0], want[0]) and not y[1].isfinite().all()


def test_output_over_input_and_other_streams():
    c = Case(6, 256, 16, 4, 128, "bf16")
    want = c.run().clone()
    s = torch.cuda.Stream()
    c.op.y = x = c.dev["x"].clone()
    s.wait_stream(torch.cuda.current_stream())
    c.run(x=x, stream=s)
    s.synchronize()
    assert torch.equal(x, want)
    # two at once, with buffers of their own
    other = Case(11, 384, 8, 2, 192, "f32", seed=5)
    want2 = other.run().clone()
    ops = [B.ForwardFew(q.p, DEV) for q in (c, other)]
    streams = [torch.cuda.Stream() for _ in ops]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, op, st in zip((c, other), ops, streams):
            q.run(op, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(ops[0].y, want) and torch.equal(ops[1].y, want2)


@pytest.mark.parametrize("act, E", [("bf16", 16), ("f32", 12), ("mxfp8", 8)])
def test_in_a_graph(act, E):
    c = Case(5, 256, E, 2, 128, act)
    c.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for i in range(4):
        c.dev["x"].copy_(torch.randn(5, 256, device=DEV))
        c.x = c.dev["x"].cpu()
        c.op.y.fill_(3)
        g.replay()
        c.check()
        got = c.op.y.clone()
        assert torch.equal(c.run(), got)


def test_the_blocks_choices():
    """Selection and gates of moe_route for the same logits; y of moe_forward within both roundings."""
    c = Case(24, 512, 32, 6, 256, "bf16", given=True)
    y = as_f64(c.run().clone())
    r = B.route(c.p, logits=c.dev["logits"])
    assert torch.equal(r["idx"], c.op.idx) and torch.allclose(r["gate"], c.op.gate, rtol=64 * U, atol=0)
    f = B.forward(c.p, c.dev["x"], packed=c.packed, logits=c.dev["logits"])
    # moe_forward rounds h and every expert's row to bfloat16 as well: normwise the block's own bar
    assert np.max(np.abs(as_f64(f["y"]) - y)) <= 2e-2 * np.max(np.abs(y))


def test_weights_past_32_bit_offsets():
    """The last of 140 experts, 4.7 GB into W1 and 2.3 GB into W2: its rows are those of the expert alone."""
    T, d, H, E = 3, 2048, 2048, 140
    one = Case(T, d, 1, 1, H, "f32", given=True)
    n1, n2 = 2 * H * d, d * H
    p = B.problem(T, d, E, 1, H, "f32", logits_given=True)
    packed = torch.zeros(B.packed_weight_bytes(p), dtype=torch.uint8, device=DEV)
    assert n1 * 4 * (E - 1) > 1 << 32
    flat, small = packed.view(torch.float32), one.packed.view(torch.float32)
    flat[(E - 1) * n1:E * n1].copy_(small[:n1])
    flat[E * n1 + (E - 1) * n2:].copy_(small[n1:])
    logits = torch.zeros(T, E, device=DEV)
    logits[:, E - 1] = 1
    op = B.ForwardFew(p, DEV)
    op(one.dev["x"], packed, logits=logits)
    want = one.run()
    # a gate of one expert is 1
    assert torch.equal(op.y, want) and (op.idx == E - 1).all()
