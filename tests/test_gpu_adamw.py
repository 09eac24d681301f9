"""The gradients' norm and the AdamW step (moe_grad_norm, moe_adamw) against their float64 oracle (marked gpu).

Tolerances, from the arithmetic (u = 2^-24, half a float32 step).  m and v are
sums of two products of which each factor is rounded to float32 (the betas, what
they leave of 1, the clipped gradient): 5 u of the summands' sizes; an 8-bit
moment's value takes two more roundings.  The step m c1 / (sqrt(v) c2 + eps)
passes through at most 10 roundings besides m's error; the weight takes one of
its own and 3 of the decay's.  Codes and bfloat16 weights are cut from a place
that these errors move: they are the oracle's where its place is further than
that from a border, else one beside it."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import training_ops as Q
from routing_dispatch_grouped_router_amd import binding as B
from routing_dispatch_grouped_router_amd.workloads import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BETAS, EPS = (0.9, 0.95), 1e-8


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


class Set:
    """Tensors of an optimizer in flat buffers with room between them that nothing may touch."""

    def __init__(self, sizes, w, g, states, seed, steps=7, scale=1.0):
        self.sizes, self.w_kind, self.states, self.seed = sizes, w, states, seed
        rng = np.random.default_rng(seed)
        total = sum(-(-n // 64) * 64 + 64 for n in sizes)
        self.at = np.cumsum([64] + [-(-n // 64) * 64 + 64 for n in sizes[:-1]])

        def flat(dtype, draw):
            out = torch.full((total + 64,), 77.0, device=DEV).to(dtype)
            return out, [self._fill(out, i, draw) for i in range(len(sizes))]
        n = rng.standard_normal
        self.flats, self.lists = {}, {}

        def make(name, dtype, draw):
            self.flats[name], self.lists[name] = flat(dtype, draw)
        make("g", _dtype(g), lambda k: scale * 1e-2 * n(k) * np.exp(n(k)))
        make("w", torch.float32 if w == "f32" else torch.bfloat16, lambda k: 0.02 * n(k))
        if w == "master":
            make("master", torch.float32, lambda k: 0.02 * n(k))
        m, r = (lambda k: scale * 3e-3 * n(k)), (lambda k: scale * 1e-2 * (0.2 + rng.random(k)))
        if states == "f32":
            make("m", torch.float32, m)
            make("v", torch.float32, lambda k: r(k) ** 2)
        else:
            for name, draw in (("m", m), ("r", r)):
                codes = []
                self.flats[name] = torch.full((total + 64,), 77, dtype=torch.uint8, device=DEV)
                self.flats[name + "_scale"] = torch.full((total,), 77.0, device=DEV)
                self.lists[name], self.lists[name + "_scale"] = [], []
                for i, k in enumerate(sizes):
                    c, s, _ = Q.encode8(draw(k), np.full(k, 32768))
                    for key, a, off in ((name, torch.from_numpy(c), self.at[i]),
                                        (name + "_scale", torch.from_numpy(s.astype(np.float32)), self.at[i] // 4)):
                        part = self.flats[key][off:off + len(a)]
                        part.copy_(a)
                        self.lists[key].append(part)
        self.step = torch.tensor([steps, 0], dtype=torch.int32, device=DEV)
        self.decay = [0.1 * (i % 3) for i in range(len(sizes))]
        self.lr_scale = [1.0 + 0.25 * (i % 2) for i in range(len(sizes))]

    def _fill(self, out, i, draw):
        part = out[self.at[i]:self.at[i] + self.sizes[i]]
        part.copy_(torch.from_numpy(draw(self.sizes[i]).astype(np.float32)))
        return part

    def optimizer(self, **kw):
        more = {k: v for k, v in self.lists.items() if k not in ("w", "g")}
        args = dict(lr=2e-3, betas=BETAS, eps=EPS, weight_decay=self.decay, lr_scale=self.lr_scale, states=self.states,
                    seed=self.seed, step=self.step)
        return B.AdamW(self.lists["w"], self.lists["g"], **{**args, **more, **kw})

    def host(self):
        return {k: [t.clone().cpu() for t in v] for k, v in self.lists.items()}

    def gaps(self):
        """What stands outside the tensors."""
        out = {}
        for k, f in self.flats.items():
            keep = torch.ones(f.numel(), dtype=torch.bool)
            for i, t in enumerate(self.lists[k]):
                off = self.at[i] // 4 if k.endswith("_scale") else self.at[i]
                keep[off:off + t.numel()] = False
            out[k] = f.cpu()[keep].float()
        return out


def _near(place, tol):
    """Whether an error of tol in a place can move it over a border."""
    return np.abs(place - np.round(place)) <= tol


def _check_codes(name, got, want, place, tol):
    got, want = got.numpy().astype(int), want.astype(int)
    off = got != want
    assert np.all(~off | (_near(place, tol) & (np.abs((got & 127) - (want & 127)) <= 1))), f"{name}: {off.sum()} codes off"


def _check_step(s: Set, before, after, t, lr, factor=1.0, eps=EPS):
    for i, n in enumerate(s.sizes):
        if n == 0:
            continue
        g = as_f64(before["g"][i]) * factor
        w = as_f64(before["master" if s.w_kind == "master" else "w"][i])
        if s.states == "f32":
            m, v, extra = as_f64(before["m"][i]), as_f64(before["v"][i]), 0
        else:
            m, v = Q.decode8(before["m"][i], before["m_scale"][i]), Q.decode8(before["r"][i], before["r_scale"][i]) ** 2
            extra = 3
        rate, decay = float(np.float32(lr)) * s.lr_scale[i], float(np.float32(s.decay[i]))
        w1, m1, v1 = Q.adamw(w, g, m, v, t, rate, BETAS, eps, decay)
        em = (5 + extra) * U * (BETAS[0] * np.abs(m) + (1 - BETAS[0]) * np.abs(g)) + 1e-45
        ev = (6 + extra) * U * v1 + 1e-45
        with np.errstate(divide="ignore", invalid="ignore"):
            den = np.sqrt(v1 / (1 - BETAS[1] ** t)) + eps
            step = np.abs(m1) / (1 - BETAS[0] ** t) / den
            rel = 10 * U + np.where(v1 > 0, ev / np.maximum(v1, 1e-300), 0)
            ew = 1.01 * (U * np.abs(w1) + rate * (step * rel + em / (1 - BETAS[0] ** t) / den + 4 * U * decay * np.abs(w)))
        bits = Q.random_bits(s.seed, t, i, n)
        if s.states == "f32":
            for name, ref, tol in (("m", m1, em), ("v", v1, ev)):
                assert np.all(np.abs(as_f64(after[name][i]) - ref) <= tol), name
        else:
            for name, ref, err, r16 in (("m", m1, em, bits & np.uint32(0xFFFF)), ("r", np.sqrt(v1), (3 + ev / np.maximum(v1, 1e-300) / U) * U * np.sqrt(v1), bits >> np.uint32(16))):
                codes, scales, place = Q.encode8(ref, r16)
                top = np.repeat(scales, 128)[:n] * 448
                worst = np.repeat([e.max() for e in np.split(err, range(128, n, 128))], 128)[:n]   # the scale's error
                rel = err / np.maximum(np.abs(ref), 1e-300) + worst / np.maximum(top, 1e-300) + 4 * U
                assert np.all(np.abs(as_f64(after[name + "_scale"][i]) - scales) <= scales * 2 * U + np.array(
                    [e.max() for e in np.split(err, range(128, n, 128))]) / 448), name
                # a place is at most 16 of its value's relative errors wide, 126 for one that is not a normal code
                _check_codes(name, after[name][i], codes, place, 16 * rel + 2.0 ** -20)
        if s.w_kind == "bf16":
            again = Q.mix(bits + np.uint32(0x7F4A7C15)) & np.uint32(0xFFFF)
            ref, place = Q.round_bf16(w1, again)
            got = as_f64(after["w"][i])
            ulp = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(w1), 2.0 ** -126))) - 7)
            off = got != ref
            assert np.all(~off | (_near(place, ew / ulp + 2.0 ** -16) & (np.abs(got - ref) <= ulp))), f"w: {off.sum()} off"
        else:
            name = "w" if s.w_kind == "f32" else "master"
            assert np.all(np.abs(as_f64(after[name][i]) - w1) <= ew), name
            if s.w_kind == "master":
                assert torch.equal(after["w"][i], after["master"][i].to(torch.bfloat16))


SIZES = [1, 7, 8, 9, 0, 127, 128, 129, 1000, 2047, 2048, 2049, 4095, 4096, 4097, 12345]


@pytest.mark.parametrize("states", ["f32", "8bit"])
@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("w", ["f32", "master", "bf16"])
def test_step(w, g, states):
    print(f"[adamw] {w} {g} {states}", flush=True)
    s = Set(SIZES, w, g, states, seed=len(w) * 100 + len(g))
    before, gaps = s.host(), s.gaps()
    op = s.optimizer()
    op()
    torch.cuda.synchronize()
    assert op.step.tolist() == [8, 0]
    after = s.host()
    _check_step(s, before, after, 8, 2e-3)
    assert all(torch.equal(a, b) for a, b in zip(before["g"], after["g"]))
    for k, v in s.gaps().items():
        assert torch.equal(v, gaps[k]), f"{k}: written outside the tensors"
    # the next, clipped
    norm = op.grad_norm(0.01)
    op(clip=norm)
    torch.cuda.synchronize()
    _check_step(s, after, s.host(), 9, 2e-3, factor=float(norm[1]))
    assert op.step.tolist() == [9, 0] and float(norm[1]) < 1


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_first_steps_from_zero(states):
    """Moments that the constructor makes; steps 1 to 3; a block of zeros; eps 0 where nothing is zero."""
    rng = np.random.default_rng(4)
    w = torch.from_numpy(rng.standard_normal(3000).astype(np.float32)).to(DEV)
    g = torch.from_numpy(rng.standard_normal(3000).astype(np.float32)).to(DEV)
    g[128:256] = 0
    op = B.AdamW([w], [g], lr=0.01, betas=BETAS, weight_decay=0.0, states=states, seed=11)
    s = Set.__new__(Set)
    s.sizes, s.w_kind, s.states, s.seed, s.decay, s.lr_scale = [3000], "f32", states, 11, [0.0], [1.0]
    s.lists = dict(w=[w], g=[g], m=op.m, **(dict(v=op.v) if states == "f32" else dict(r=op.r, m_scale=op.m_scale, r_scale=op.r_scale)))
    for t in (1, 2, 3):
        before = s.host()
        op()
        torch.cuda.synchronize()
        after = s.host()
        _check_step(s, before, after, t, 0.01)
        assert torch.equal(after["w"][0][128:256], before["w"][0][128:256])
    assert op.step.tolist() == [3, 0]


def test_kinds_together_count_one_step():
    """Tensors of several kinds in one list, as a block's weights (bf16 with a master) and a norm's (float32)."""
    parts = [Set([300, 5000], "f32", "f32", "f32", 1), Set([700], "master", "bf16", "f32", 2), Set([4100], "bf16", "f32", "f32", 3)]
    weights, grads, master, m, v = [], [], [], [], []
    for s in parts:
        weights += s.lists["w"]
        grads += s.lists["g"]
        master += s.lists.get("master", [None] * len(s.sizes))
        m += s.lists["m"]
        v += s.lists["v"]
    step = torch.tensor([4, 0], dtype=torch.int32, device=DEV)
    op = B.AdamW(weights, grads, lr=2e-3, betas=BETAS, eps=EPS, weight_decay=0.1, master=master, m=m, v=v, step=step, seed=5)
    before = [s.host() for s in parts]
    op()
    torch.cuda.synchronize()
    assert step.tolist() == [5, 0]
    first = 0
    for s, b in zip(parts, before):
        s.decay, s.lr_scale = [0.1] * len(s.sizes), [1.0] * len(s.sizes)
        if s.w_kind != "bf16":
            _check_step(s, b, s.host(), 5, 2e-3)
        else:   # its place in the list is part of the random bits
            s.seed = 5
            pad = Set.__new__(Set)
            pad.__dict__.update(s.__dict__)
            pad.sizes = [0] * first + s.sizes
            pad.decay, pad.lr_scale = [0.1] * len(pad.sizes), [1.0] * len(pad.sizes)
            _check_step(pad, {k: [None] * first + t for k, t in b.items()}, {k: [None] * first + t for k, t in s.host().items()}, 5, 2e-3)
        first += len(s.sizes)


def test_a_norm_that_is_not_finite_leaves_everything():
    for bad in (float("nan"), float("inf")):
        s = Set([5000, 130], "master", "f32", "8bit", 6)
        s.lists["g"][1][3] = bad
        op = s.optimizer()
        before = {k: f.clone() for k, f in s.flats.items()}
        norm = op.grad_norm(1.0)
        op(clip=norm)
        torch.cuda.synchronize()
        assert norm[1].isnan() and not norm[0].isfinite() and op.step.tolist() == [7, 0]
        assert all(torch.equal(f.view(torch.uint8), before[k].view(torch.uint8)) for k, f in s.flats.items())
        s.lists["g"][1][3] = 0.5          # and the next step is made
        op(clip=op.grad_norm(1.0))
        assert op.step.tolist() == [8, 0]


def test_8bit_moments_of_elements_that_are_not_finite():
    """Without clipping, a NaN or infinite gradient is its element's, not its block's."""
    s = Set([1000], "f32", "f32", "8bit", 8)
    clean = s.host()
    s.lists["g"][0][200], s.lists["g"][0][300] = float("nan"), float("inf")
    op = s.optimizer()
    op()
    m, r, w = s.lists["m"][0].cpu(), s.lists["r"][0].cpu(), s.lists["w"][0].cpu()
    assert (m[200] & 127) == 127 and (r[200] & 127) == 127 and (m[300] & 127) == 127 and (r[300] & 127) == 127
    assert w[200].isnan()
    keep = np.ones(1000, bool)
    keep[[200, 300]] = False
    assert np.isfinite(Q.decode8(m, s.lists["m_scale"][0].cpu())[keep]).all() and w[torch.from_numpy(keep)].isfinite().all()
    assert not torch.equal(w[:200], clean["w"][0][:200])


@pytest.mark.parametrize("scale", [1e-24, 1e15])
def test_gradients_of_extreme_sizes(scale):
    """Squares at float32's ends: v of denormal or huge values, roots and steps as the formula has them."""
    s = Set([3000], "f32", "f32", "f32", 9, scale=scale)
    before = s.host()
    s.optimizer(eps=1e-30 if scale < 1 else EPS)()
    torch.cuda.synchronize()
    after = s.host()
    g, m, v = (as_f64(before[k][0]) for k in ("g", "m", "v"))
    _, m1, v1 = Q.adamw(0, g, m, v, 8, 0, BETAS, EPS, 0)
    assert np.all(np.abs(as_f64(after["m"][0]) - m1) <= 6 * U * (np.abs(m) + np.abs(g)) + 1e-45)
    assert np.all(np.abs(as_f64(after["v"][0]) - v1) <= 8 * U * v1 + 3 * 2.0 ** -149)   # denormal products
    assert after["w"][0].isfinite().all()


@pytest.mark.parametrize("g", ["f32", "bf16"])
def test_grad_norm(g):
    for sizes in ([1], [0, 3], SIZES, [3_000_001, 17, 5_000_000]):
        print(f"[grad norm] {sizes[:3]} {g}", flush=True)
        rng = np.random.default_rng(len(sizes))
        grads = [torch.from_numpy((rng.standard_normal(n) * 10 ** rng.uniform(-6, 2)).astype(np.float32)).to(DEV).to(_dtype(g)) for n in sizes]
        op = B.GradNorm(grads)
        for most in (1e-3, 1.0, float("inf")):
            norm, factor = Q.grad_norm([as_f64(t) for t in grads], most)
            first = op(most).clone()
            assert torch.equal(first, op(most))
            got = as_f64(first)
            # float64 sums and root, one rounding; of the factor also that of max_norm, a float32 argument
            assert abs(got[0] - norm) <= U * norm * (1 + 1e-6) and abs(got[1] - factor) <= 2 * U * factor * (1 + 1e-6)


def test_grad_norm_of_large_values_and_of_none():
    a = torch.full((1000,), 3e38, device=DEV)
    norm = B.GradNorm([a])(1.0)
    # past float32, not past the sum; the factor, 1.054e-40, is a denormal: half a step of 2^-149 is 6.7e-6 of it
    assert norm[0].isinf() and abs(float(norm[1]) * 3e38 * 1000 ** 0.5 - 1) < 7e-6
    b = torch.full((100,), 1e-30, device=DEV)
    assert abs(float(B.GradNorm([b])()[0]) / 1e-29 - 1) < 1e-6
    zero = B.GradNorm([torch.zeros(5, device=DEV), torch.empty(0, device=DEV)])(2.0)
    assert zero.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_steps_in_a_graph(states):
    """Replays take the next step each, as eager steps do, with the learning rate of the time."""
    sizes = [5000, 129, 70_000]
    eager, graphed = (Set(sizes, "bf16", "f32", states, 21) for _ in range(2))
    a, b = eager.optimizer(), graphed.optimizer()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        b(clip=b.grad_norm(0.5))
    for i in range(4):
        a.lr.fill_(1e-3 * (i + 1))
        b.lr.fill_(1e-3 * (i + 1))
        a(clip=a.grad_norm(0.5))
        scratch = torch.randn(4096, device=DEV)
        g.replay()
        torch.cuda.synchronize()
        for k in eager.flats:
            assert torch.equal(eager.flats[k], graphed.flats[k]), (i, k)
        assert a.step.tolist() == b.step.tolist() == [8 + i, 0] and torch.equal(a.norm, b.norm)
        del scratch


def test_two_optimizers_at_once():
    sizes = [300_000, 77, 4097]
    sets = [Set(sizes, "master", "f32", "f32", 31), Set(sizes, "bf16", "bf16", "8bit", 32)]
    twins = [Set(sizes, "master", "f32", "f32", 31), Set(sizes, "bf16", "bf16", "8bit", 32)]
    for t in twins:
        op = t.optimizer()
        for _ in range(3):
            op(clip=op.grad_norm(1.0))
    torch.cuda.synchronize()
    ops, streams = [s.optimizer() for s in sets], [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for op, st in zip(ops, streams):
            op(clip=op.grad_norm(1.0, stream=st), stream=st)
    torch.cuda.synchronize()
    for s, t in zip(sets, twins):
        assert all(torch.equal(s.flats[k], t.flats[k]) for k in s.flats)


def test_refusals():
    w, g = torch.zeros(256, device=DEV), torch.zeros(256, device=DEV)
    B.AdamW([w], [g])
    with pytest.raises(B.MoeError, match="status -7"):
        B.AdamW([w, w], [g, g])                                  # the same weight twice
    with pytest.raises(B.MoeError, match="status -7"):
        B.AdamW([w], [w])                                        # a gradient that is a weight
    with pytest.raises(B.MoeError, match="status -7"):
        B.AdamW([w[1:]], [g[1:]])                                # not aligned
    with pytest.raises(B.MoeError, match="status -3"):
        B.AdamW([w], [g], master=[w.clone()])                    # a master of float32 weights
    B.AdamW([w, w.clone()], [g, g])                              # two weights of one gradient
    with pytest.raises(ValueError, match="contiguous"):
        B.AdamW([w.view(16, 16).t()], [g.view(16, 16)])
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        B.AdamW([w.half()], [g])
    with pytest.raises(ValueError, match="grads: expected"):
        B.AdamW([w], [g[:5]])
    with pytest.raises(ValueError, match="device tensor"):
        B.AdamW([w], [g.cpu()])
    op = B.AdamW([w], [g])
    for name in ("m", "v", "weights", "grads", "lr", "norm", "step", "states"):
        with pytest.raises(AttributeError):
            setattr(op, name, None)
    with pytest.raises(TypeError):
        op.m[0] = w
    op = B.AdamW([w], [g], betas=(1.0, 0.9))
    with pytest.raises(B.MoeError, match="status -7"):
        op()
    for most in (0.0, -1.0, float("nan")):
        with pytest.raises(B.MoeError, match="status -7"):
            op.grad_norm(most)
    norm_only = B.GradNorm([g])
    hyper = B.AdamwHyper(0.9, 0.9, 1e-8, 0)
    assert B.lib().moe_adamw(norm_only._plan_p, norm_only._table_p, ctypes.byref(hyper), w.data_ptr(), None, g.data_ptr(), None) == -6
