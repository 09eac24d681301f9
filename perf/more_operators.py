"""Operators of training the routed block and of trying it, as cases that can be timed and compared.

``own`` False: the plain form of each operator, elementary torch operations in
32 bits, rounded once where a result is stored.  ``own`` True: the library's
calls.  Both take the state that ``prepare`` makes, and return the same outputs.

Operators (the field ``op`` of a case):
  layer_norm           layer norm with the residual's addition; for act "mxfp8"
                       the MXFP8 codes and scales of the rows as well
  layer_norm_backward  its gradients
  grad_norm            the norm of many gradient tensors and the factor that clips them
  adamw                one AdamW step over many tensors, with or without that clipping;
                       the moments in 32 bits or in 8
  few                  the block for a few tokens, router included, on the packed weights
                       that the block's forward takes

The tensors of an optimizer lie in flat buffers, each at a multiple of 128
elements, so that the buffers are the outputs.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-5
BETA1, BETA2, ADAM_EPS, MAX_NORM = 0.9, 0.99, 1e-8, 1.0
BLOCK = 128            # elements of an 8-bit moment that share a scale


def listed():
    return [
        # one token being generated: latency is all there is
        dict(name="layer_norm_one_token", op="layer_norm", act="bf16", T=1, d=4096, residual=True),
        # the rows of the largest MXFP8 block, codes for its experts and bf16 rows for its router
        dict(name="layer_norm_rows_mxfp8", op="layer_norm", act="mxfp8", T=32768, d=2048, residual=True),
        # training, the rows of the largest bf16 block
        dict(name="layer_norm_bwd_bf16", op="layer_norm_backward", act="bf16", T=16384, d=4096, residual=True),
        # training, an odd small float32 batch
        dict(name="layer_norm_bwd_odd_f32", op="layer_norm_backward", act="f32", T=777, d=192, residual=False),
        # the gradients of the 8-expert block: three large tensors, the router, a norm
        dict(name="grad_norm_block", op="grad_norm", set="block", E=8, d=2048, H=1024, g="f32"),
        # many odd tensors, most of them small
        dict(name="grad_norm_odd", op="grad_norm", set="odd", count=60, largest=20000, g="bf16"),
        # mixed precision as the block trains: bf16 weights, float32 masters and moments, clipped
        dict(name="adamw_block", op="adamw", set="block", E=8, d=2048, H=1024, w="master", g="f32", states="f32", clip=True),
        # the least memory: bf16 weights without masters, 8-bit moments
        dict(name="adamw_block_8bit", op="adamw", set="block", E=8, d=2048, H=1024, w="bf16", g="f32", states="8bit", clip=False),
        # many odd float32 tensors, most of them small: launches count
        dict(name="adamw_odd", op="adamw", set="odd", count=60, largest=20000, w="f32", g="f32", states="f32", clip=False),
        # one token of the 64-expert block
        dict(name="few_t1", op="few", act="bf16", T=1, d=4096, E=64, k=8, H=1536, padded=0),
        # a ragged small batch (its last tokens padding) on the MXFP8 block's weights
        dict(name="few_t7_mxfp8", op="few", act="mxfp8", T=7, d=2048, E=128, k=4, H=1024, padded=2),
        # several rows an expert
        dict(name="few_t16_e8", op="few", act="bf16", T=16, d=2048, E=8, k=4, H=1024, padded=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_backward", "grad_norm", "adamw", "adamw", "few", "few"])
    if op in ("layer_norm", "layer_norm_backward"):
        act = rng.choice(["bf16", "bf16", "f32"] + (["mxfp8", "mxfp8"] if op == "layer_norm" else []))
        unit = 128 if act == "mxfp8" else 64
        d = unit * _log(rng, 1, 8192 // unit)
        T = _log(rng, 1, min(32768, (1 << 26) // (d * (2 if act == "f32" else 1))))
        return dict(op=op, act=act, T=T, d=d, residual=rng.random() < 0.7)
    if op in ("grad_norm", "adamw"):
        c = dict(op=op, g=rng.choice(["f32", "f32", "bf16"]))
        if rng.random() < 0.5:
            d, H = 64 * _log(rng, 1, 32), 64 * _log(rng, 1, 24)
            c.update(set="block", E=min(_log(rng, 1, 64), (1 << 24) // (d * H)), d=d, H=H)
        else:
            c.update(set="odd", count=_log(rng, 1, 200), largest=_log(rng, 2, 200000))
        if op == "adamw":
            c.update(w=rng.choice(["f32", "master", "bf16"]), states=rng.choice(["f32", "8bit"]), clip=rng.random() < 0.5)
        return c
    act = rng.choice(["bf16", "bf16", "mxfp8", "f32"])
    unit = 64 if act != "mxfp8" else 128
    d, H = unit * _log(rng, 1, 4096 // unit), unit * _log(rng, 1, 2048 // unit)
    E = max(1, min(_log(rng, 1, 128), (3 << (27 if act != "f32" else 26)) // (d * H)))
    T = _log(rng, 1, 32)
    return dict(op=op, act=act, T=T, d=d, E=E, k=rng.randint(1, min(E, 8)), H=H, padded=rng.choice([0, rng.randint(0, T // 2)]))


# ----------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _store(act):
    return torch.float32 if act == "f32" else torch.bfloat16


def prepare(case, seed):
    g = _gen(seed)
    return dict(case=case, **globals()["_inputs_" + case["op"]](case, g))


def _activations(c, g):
    """N(0.3, 1) rows in which one value in a hundred is 64 times larger, as residual streams have them."""
    x = 0.3 + _randn(g, c["T"], c["d"])
    big = torch.rand(c["T"], c["d"], generator=g, device=DEV) < 0.01
    return torch.where(big, x * 64, x).to(_store(c["act"]))


def _inputs_layer_norm(c, g):
    return dict(x=_activations(c, g), residual=_randn(g, c["T"], c["d"]).to(_store(c["act"])) if c["residual"] else None,
                weight=(1 + 0.1 * _randn(g, c["d"])).to(_store(c["act"])), bias=(0.1 * _randn(g, c["d"])).to(_store(c["act"])))


def _inputs_layer_norm_backward(c, g):
    dt = _store(c["act"])
    s = _activations(c, g)
    mean = s.double().mean(1)
    rstd = ((s.double() - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
    return dict(s=s, mean=mean.float(), rstd=rstd, dy=(0.01 * _randn(g, c["T"], c["d"])).to(dt),
                dsum=(0.01 * _randn(g, c["T"], c["d"])).to(dt) if c["residual"] else None,
                weight=(1 + 0.1 * _randn(g, c["d"])).to(dt))


def _sizes(c):
    """Elements of each tensor, and its weight decay."""
    if c["set"] == "block":      # gate, up and down projections, the router; weight and bias of a norm
        n = [c["E"] * c["d"] * c["H"]] * 3 + [c["d"] * c["E"], c["d"], c["d"]]
        return n, [0.1] * 4 + [0.0] * 2
    r = random.Random(c["count"] * 1000003 + c["largest"])
    n = [_log(r, 1, c["largest"]) for _ in range(c["count"])]
    return n, [0.1 * (i % 2) for i in range(len(n))]


def _flat(c):
    """Where each tensor begins in a flat buffer, its size and weight decay, and the buffer's size."""
    n, decay = _sizes(c)
    room = [-(-v // BLOCK) * BLOCK for v in n]
    at = [sum(room[:i]) for i in range(len(room))]
    return list(zip(at, n, decay)), sum(room)


def _gradients(c, g, parts, total):
    """Tensors of different scale; some values far out."""
    x = _randn(g, total) * torch.exp(_randn(g, total // BLOCK)).repeat_interleave(BLOCK) * 1e-3
    used = torch.zeros(total, dtype=torch.bool, device=DEV)
    for at, n, _ in parts:
        used[at:at + n] = True
    return torch.where(used, x, 0.0).to(torch.float32 if c["g"] == "f32" else torch.bfloat16), used


def _inputs_grad_norm(c, g):
    parts, total = _flat(c)
    return dict(parts=parts, g=_gradients(c, g, parts, total)[0])


def _inputs_adamw(c, g):
    parts, total = _flat(c)
    grad, used = _gradients(c, g, parts, total)
    w = torch.where(used, 0.02 * _randn(g, total), 0.0)
    s = dict(parts=parts, g=grad, w=w if c["w"] == "f32" else w.bfloat16(), master=w if c["w"] == "master" else None)
    m = torch.where(used, 0.3 * _randn(g, total) * grad.float().abs().mean(), 0.0)
    r = torch.where(used, (0.5 + torch.rand(total, generator=g, device=DEV)) * grad.float().abs().mean(), 0.0)
    if c["states"] == "8bit":
        s["m"], s["m_scale"] = _nearest8(m)
        s["r"], s["r_scale"] = _nearest8(r)
    else:
        s["m"], s["v"] = m, r * r
    # elements of a tensor's blocks carry the tensor's number, decay and the block's number in it
    room = torch.tensor([-(-n // BLOCK) for _, n, _ in parts], device=DEV)
    first = torch.cumsum(room, 0) - room
    s["tensor"] = torch.arange(len(parts), device=DEV).repeat_interleave(room)
    s["block"] = torch.arange(total // BLOCK, device=DEV) - first[s["tensor"]]
    s["decay"] = torch.tensor([d for _, _, d in parts], device=DEV)[s["tensor"]].repeat_interleave(BLOCK)
    s["lr"] = torch.tensor([3e-4], device=DEV)
    s["step"] = torch.tensor([int(torch.randint(1, 2000, (1,), generator=g, device=DEV)), 0], dtype=torch.int32, device=DEV)
    s["seed"] = int(torch.randint(0, 1 << 30, (1,), generator=g, device=DEV))
    return s


def _nearest8(x):
    """Codes and scales of the nearest E4M3 values."""
    b = x.view(-1, BLOCK)
    scale = b.abs().amax(1) / 448
    q = (b / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(-1), scale


def _quantize_mxfp8(b):
    """E4M3 codes and scale bytes of b [n, K] in blocks of 32 columns."""
    v = b.view(b.shape[0], -1, 32)
    amax = v.abs().amax(2)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 8, -127).clamp(-127, 127)
    q = torch.ldexp(v, -e[:, :, None].float()).clamp(-448, 448)
    return q.view(b.shape).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _inputs_few(c, g):
    """The packed weights are one buffer: W1 [E, 2H, d] (rows: 32 gate, 32 up, ...) and W2 [E, d, H], for MXFP8 with the
    scales S1 [E, d/128, 2H, 4] and S2 [E, H/128, d, 4]."""
    T, d, E, H = (c[n] for n in ("T", "d", "E", "H"))
    mx, dt = c["act"] == "mxfp8", _store(c["act"])
    packed = torch.empty(E * 3 * d * H * 33 // 32 if mx else E * 3 * d * H * dt.itemsize, dtype=torch.uint8, device=DEV)
    w1, w2, s1, s2 = _split_packed(packed, c)
    for e in range(E):
        for w, sc, rows, K in ((w1, s1, 2 * H, d), (w2, s2, d, H)):
            v = 0.02 * _randn(g, rows, K)
            if mx:
                w[e], q = _quantize_mxfp8(v)
                sc[e] = q.view(rows, K // 128, 4).transpose(0, 1)
            else:
                w[e] = v
    mask = None
    if c["padded"]:
        mask = torch.ones(T, dtype=torch.uint8, device=DEV)
        mask[T - c["padded"]:] = 0
    return dict(x=_randn(g, T, d).to(dt), w_router=(0.02 * _randn(g, d, E)).to(dt), mask=mask, packed=packed)


def _split_packed(packed, c):
    d, E, H = c["d"], c["E"], c["H"]
    n = E * d * H
    if c["act"] != "mxfp8":
        w = packed.view(_store(c["act"]))
        return w[:2 * n].view(E, 2 * H, d), w[2 * n:].view(E, d, H), None, None
    w1, w2, s1, s2 = packed.split([2 * n, n, 2 * n // 32, n // 32])
    return w1.view(E, 2 * H, d), w2.view(E, d, H), s1.view(E, d // 128, 2 * H, 4), s2.view(E, H // 128, d, 4)


# ----------------------------------------------------------------------------- one pass


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _plain_layer_norm(s):
    c, dt = s["case"], s["x"].dtype
    t = s["x"].float()
    if s["residual"] is not None:
        t = t + s["residual"].float()
    mean = t.mean(1)
    n = t - mean[:, None]
    rstd = torch.rsqrt((n * n).mean(1) + EPS)
    y = (n * rstd[:, None] * s["weight"].float() + s["bias"].float()).to(dt)
    out = dict(y=y, mean=mean, rstd=rstd)
    if s["residual"] is not None:
        out["sum"] = t.to(dt)
    if c["act"] == "mxfp8":   # the codes are those of the stored row, so that they are what the block would make of it
        q, scale = _quantize_mxfp8(y.float())
        out["q"] = q.view(torch.float8_e4m3fn)
        out["q_scale"] = scale.view(torch.float8_e8m0fnu)
    return out


def _plain_layer_norm_backward(s):
    n, dy, rstd = (s["s"].float() - s["mean"][:, None]) * s["rstd"][:, None], s["dy"].float(), s["rstd"][:, None]
    u = dy * s["weight"].float()
    ds = rstd * (u - u.mean(1, keepdim=True) - n * (u * n).mean(1, keepdim=True))
    if s["dsum"] is not None:
        ds = ds + s["dsum"].float()
    return dict(ds=ds.to(s["s"].dtype), dweight=(dy * n).sum(0), dbias=dy.sum(0))


def _plain_norm_of(g):
    """float32 [2]: the norm of every gradient together, and the factor that brings it to MAX_NORM at most."""
    norm = g.double().square().sum().sqrt()
    return torch.stack([norm, torch.where(norm > MAX_NORM, MAX_NORM / norm, 1.0)]).float()


def _plain_grad_norm(s):
    return _plain_norm_of(s["g"])


_LOW = 0xFFFFFFFF


def _mix(h):
    """The finalizer of MurmurHash3 (32 bits) of int64 tensors that hold 32-bit values."""
    h = (h ^ (h >> 16)) * 0x85EBCA6B & _LOW
    h = (h ^ (h >> 13)) * 0xC2B2AE35 & _LOW
    return h ^ (h >> 16)


def _hashes(s, t):
    """A 32-bit number for every element: of the seed, the step, the tensor, the block in it and the element in that."""
    key = _mix((_mix(_mix(t.long()) ^ s["seed"]) + s["tensor"]) & _LOW)
    key = _mix(key ^ s["block"])
    return _mix((key[:, None] + torch.arange(BLOCK, device=DEV) * 0x9E3779B9) & _LOW)


def _round8(x, r16):
    """E4M3 codes and block scales of x [blocks, BLOCK], rounded up where the 16 random bits say so."""
    amax = x.abs().amax(1)
    amax = torch.where(amax < 2.0 ** -100, 0.0, amax)
    a = (x.abs() * torch.where(amax > 0, 448 / amax, 0.0)[:, None]).clamp(max=448)
    u = (a * 2.0 ** -120).view(torch.int32)          # E4M3's exponent and fraction above 20 more bits
    code = ((u + (r16.int() * 16 + 8)) >> 20).clamp(max=0x7E)
    return (code | ((x < 0).int() << 7)).to(torch.uint8).view(-1), amax / 448


def _plain_adamw(s):
    c = s["case"]
    out = {}
    g = s["g"].float()
    if c["clip"]:
        out["norm"] = _plain_norm_of(s["g"])
        g = g * out["norm"][1]
    s["step"][0] += 1
    t = s["step"][0]
    if c["states"] == "8bit":
        h = _hashes(s, t)
        m = (s["m"].view(torch.float8_e4m3fn).float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        r = (s["r"].view(torch.float8_e4m3fn).float().view(-1, BLOCK) * s["r_scale"][:, None]).view(-1)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    c1, c2 = ((1 - torch.pow(torch.tensor(b, dtype=torch.float64, device=DEV), t)).float() for b in (BETA1, BETA2))
    w = s["w"].float() if s["master"] is None else s["master"]
    w = w - s["lr"] * ((m / c1) / ((v / c2).sqrt() + ADAM_EPS) + s["decay"] * w)
    if c["w"] == "bf16":       # rounded up where 16 random bits say so: a step is smaller than a bf16 weight's last bit
        r16 = _mix((_hashes(s, t) + 0x7F4A7C15) & _LOW).view(-1) & 0xFFFF
        s["w"].copy_(((w.view(torch.int32) + r16.int()) & -65536).view(torch.float32))
    else:
        s["w"].copy_(w)
    if s["master"] is not None:
        s["master"].copy_(w)
    if c["states"] == "8bit":
        for name, x, bits in (("m", m, h & 0xFFFF), ("r", v.sqrt(), h >> 16)):
            q, scale = _round8(x.view(-1, BLOCK), bits)
            s[name].copy_(q)
            s[name + "_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _state(s, out)


def _state(s, out):
    """Weights, moments and the number of steps after the step."""
    out.update(w=s["w"], master=s["master"], step=s["step"])
    if s["case"]["states"] == "8bit":
        out.update(m=s["m"].view(torch.float8_e4m3fn), r=s["r"].view(torch.float8_e4m3fn), m_scale=s["m_scale"], r_scale=s["r_scale"])
    else:
        out.update(m=s["m"], v=s["v"])
    return out


def _values(w, scale):
    """float32 [..., K] of packed weights [..., K], with MXFP8's scales [..., K/128, rows, 4]."""
    if scale is None:
        return w.float()
    e = scale.transpose(-3, -2).reshape(*w.shape[:-1], -1, 1).float() - 127
    return torch.ldexp(w.view(torch.float8_e4m3fn).float().view(*w.shape[:-1], -1, 32), e).view(w.shape)


def _plain_few(s):
    c = s["case"]
    T, d, E, k, H = (c[n] for n in ("T", "d", "E", "k", "H"))
    R = T * k
    w1, w2, s1, s2 = _split_packed(s["packed"], c)
    x = s["x"].float()
    logits = x @ s["w_router"].float()
    val, idx = torch.sort(logits, stable=True, dim=1, descending=True)
    val, idx = val[:, :k], idx[:, :k]
    z = torch.exp(val - val[:, :1])
    gate = z / z.sum(1, keepdim=True)
    at = idx.reshape(-1)
    silu = torch.nn.functional.silu
    if R <= E:      # the experts of each row, gathered
        a = (_values(w1[at], None if s1 is None else s1[at]) * x.repeat_interleave(k, 0)[:, None, :]).sum(2).view(R, H // 32, 2, 32)
        h = (silu(a[:, :, 0]) * a[:, :, 1]).reshape(R, H)
        ye = (_values(w2[at], None if s2 is None else s2[at]) * h[:, None, :]).sum(2)
    else:           # every expert on every token, and of that the rows that were asked for
        a = (x @ _values(w1, s1).view(E * 2 * H, d).t()).view(T, E, H // 32, 2, 32)
        h = (silu(a[:, :, :, 0]) * a[:, :, :, 1]).reshape(T, E, H).transpose(0, 1).contiguous()
        all_y = torch.bmm(h, _values(w2, s2).transpose(1, 2).contiguous())
        ye = all_y[at, torch.arange(R, device=x.device) // k]
    if s["mask"] is not None:
        live = s["mask"][:, None] != 0
        idx, gate = torch.where(live, idx, -1), torch.where(live, gate, 0.0)
    y = (gate[:, :, None] * ye.view(T, k, d)).sum(1)
    return dict(y=y.to(s["x"].dtype), logits=logits, idx=idx.int(), gate=gate)


# ----------------------------------------------------------------------------- the library's calls


def _handle(s, make):
    """The preallocated buffers that a program keeps from step to step."""
    if "handle" not in s:
        from routing_dispatch_grouped_router_amd import binding
        s["handle"] = make(binding)
    return s["handle"]


def _own_layer_norm(s):
    c = s["case"]
    op = _handle(s, lambda B: B.LayerNorm(B.problem(c["T"], c["d"], 1, 1, 128, c["act"]), DEV, eps=EPS, residual=c["residual"]))
    op(s["x"], s["weight"], s["bias"], residual=s["residual"])
    out = dict(y=op.y, mean=op.mean, rstd=op.rstd)
    if c["residual"]:
        out["sum"] = op.sum
    if c["act"] == "mxfp8":
        out["q"] = op.q.view(torch.float8_e4m3fn)
        out["q_scale"] = op.q_scale.view(torch.float8_e8m0fnu)
    return out


def _own_layer_norm_backward(s):
    c = s["case"]
    op = _handle(s, lambda B: B.LayerNormBackward(B.problem(c["T"], c["d"], 1, 1, 128, c["act"]), DEV))
    return op(s["dy"], s["s"], s["weight"], s["mean"], s["rstd"], dsum=s["dsum"])


def _parts(s, flat):
    return None if flat is None else [flat[at:at + n] for at, n, _ in s["parts"]]


def _scales(s, flat):
    return [flat[at // BLOCK:-(-(at + n) // BLOCK)] for at, n, _ in s["parts"]]


def _own_grad_norm(s):
    op = _handle(s, lambda B: B.GradNorm(_parts(s, s["g"])))
    return op(MAX_NORM)


def _make_adamw(B, s):
    more = dict(m=_parts(s, s["m"]))
    if s["case"]["states"] == "8bit":
        more.update(r=_parts(s, s["r"]), m_scale=_scales(s, s["m_scale"]), r_scale=_scales(s, s["r_scale"]))
    else:
        more.update(v=_parts(s, s["v"]))
    return B.AdamW(_parts(s, s["w"]), _parts(s, s["g"]), lr=s["lr"], betas=(BETA1, BETA2), eps=ADAM_EPS,
                   weight_decay=[d for _, _, d in s["parts"]], master=_parts(s, s["master"]), states=s["case"]["states"],
                   seed=s["seed"], step=s["step"], **more)


def _own_adamw(s):
    op = _handle(s, lambda B: _make_adamw(B, s))
    out = {}
    if s["case"]["clip"]:
        out["norm"] = op.grad_norm(MAX_NORM)
    op(clip=out.get("norm"))
    return _state(s, out)


def _own_few(s):
    c = s["case"]
    op = _handle(s, lambda B: B.ForwardFew(B.problem(c["T"], c["d"], c["E"], c["k"], c["H"], c["act"]), DEV))
    op(s["x"], s["packed"], w_router=s["w_router"], mask=s["mask"])
    return dict(y=op.y, logits=op.logits, idx=op.idx, gate=op.gate)


# ----------------------------------------------------------------------------- what a pass needs


def work(case):
    c = case
    b = 4 if c.get("act") == "f32" else 2
    if c["op"] == "layer_norm":
        n = c["T"] * c["d"]
        rows = n * b * (4 if c["residual"] else 2)      # x, y and with a residual that and the sum
        return dict(bytes=rows + 2 * c["d"] * b + 8 * c["T"] + (n * 33 // 32 if c["act"] == "mxfp8" else 0), flops=8 * n)
    if c["op"] == "layer_norm_backward":
        n = c["T"] * c["d"]
        return dict(bytes=n * b * (4 if c["residual"] else 3) + c["d"] * (b + 8) + 8 * c["T"], flops=13 * n)
    if c["op"] in ("grad_norm", "adamw"):
        n = sum(_sizes(c)[0])
        gb = 4 if c["g"] == "f32" else 2
        if c["op"] == "grad_norm":
            return dict(bytes=n * gb + 8, flops=2 * n)
        wb = dict(f32=8, master=10, bf16=4)[c["w"]]
        return dict(bytes=int(n * (gb + wb + (4 + 16 / BLOCK if c["states"] == "8bit" else 16))), flops=15 * n)
    live = c["T"] - c["padded"]
    used = c["E"] * (1 - (1 - c["k"] / c["E"]) ** live)   # distinct experts of evenly routed tokens
    wb = 33 / 32 if c["act"] == "mxfp8" else b
    return dict(bytes=int(used * 3 * c["d"] * c["H"] * wb) + c["d"] * c["E"] * b + 2 * b * c["T"] * c["d"] + 4 * c["T"] * (c["E"] + 2 * c["k"]),
                flops=6 * live * c["k"] * c["d"] * c["H"] + 2 * c["T"] * c["d"] * c["E"])


# ----------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    """What run() returns, from the definitions, in float64.  Values that are stored in fewer bits on the way to an
    8-bit output are rounded there, and stochastic roundings take place, since the outputs are defined by them."""
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, s)


def _exact_layer_norm(c, s):
    t = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
    mean = torch.sum(t, 1) / c["d"]
    var = torch.sum(t * t, 1) / c["d"] - mean * mean
    rstd = 1 / torch.sqrt(var + EPS)
    y = t * (rstd[:, None] * s["weight"].double()) + (s["bias"].double() - (mean * rstd)[:, None] * s["weight"].double())
    out = dict(y=y, mean=mean, rstd=rstd)
    if s["residual"] is not None:
        out["sum"] = t
    if c["act"] == "mxfp8":
        blk = y.to(torch.bfloat16).double().reshape(-1, 32)
        top = blk.abs().max(1, keepdim=True).values
        ex = torch.floor(torch.log2(torch.clamp(top, min=2.0 ** -140))).clamp(min=-119) - 8
        v = (blk / 2 ** ex).clamp(-448, 448)
        quantum = 2 ** (torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        out["q"] = (torch.round(v / quantum) * quantum).reshape(c["T"], c["d"])
        out["q_scale"] = (2 ** ex).reshape(c["T"], c["d"] // 32)
    return out


def _exact_layer_norm_backward(c, s):
    t, dy, w, mu, r = (s[n].double() for n in ("s", "dy", "weight", "mean", "rstd"))
    t = t - mu[:, None]
    plain, inner = torch.sum(dy * w, 1) / c["d"], torch.sum(t * dy * w, 1) / c["d"]
    ds = r[:, None] * dy * w - (r * plain)[:, None] - (r ** 3 * inner)[:, None] * t
    if s["dsum"] is not None:
        ds = ds + s["dsum"].double()
    return dict(ds=ds, dweight=torch.sum(t * dy * r[:, None], 0), dbias=torch.sum(dy, 0))


def _exact_grad_norm(c, s):
    n = math.sqrt(sum(float((s["g"][at:at + n].double() ** 2).sum()) for at, n, _ in s["parts"]))
    return torch.tensor([n, min(1.0, MAX_NORM / n) if n else 1.0], dtype=torch.float64, device=DEV)


def _exact_adamw(c, s):
    steps = int(s["step"][0]) + 1
    out = dict(step=torch.tensor([steps, 0], dtype=torch.int32, device=DEV))
    factor = 1.0
    if c["clip"]:
        out["norm"] = _exact_grad_norm(c, s)
        factor = float(out["norm"][1])
    eight = c["states"] == "8bit"
    old = s["w"] if s["master"] is None else s["master"]
    names = ["w"] + (["m", "r", "m_scale", "r_scale"] if eight else ["m", "v"]) + (["master"] if s["master"] is not None else [])
    for name in names:
        out[name] = torch.zeros_like(s[name], dtype=torch.float64)
    for i, (at, n, decay) in enumerate(s["parts"]):
        lo, hi = at // BLOCK, -(-(at + n) // BLOCK)
        el, bl = slice(lo * BLOCK, hi * BLOCK), slice(lo, hi)
        grad = s["g"][el].double() * factor
        code = [s[q][el].view(torch.float8_e4m3fn).double() * s[q + "_scale"][bl].double().repeat_interleave(BLOCK) if eight else s[q][el].double()
                for q in (("m", "r") if eight else ("m", "v"))]
        m = code[0] + (1 - BETA1) * (grad - code[0])
        v0 = code[1] ** 2 if eight else code[1]
        v = v0 + (1 - BETA2) * (grad * grad - v0)
        rate = float(s["lr"])
        w = old[el].double() * (1 - rate * float(torch.tensor(decay))) - rate * m / (1 - BETA1 ** steps) / (torch.sqrt(v / (1 - BETA2 ** steps)) + ADAM_EPS)
        if eight or c["w"] == "bf16":
            numbers = _exact_hash(s["seed"], steps, i, hi - lo)
        if c["w"] == "bf16":
            again = _exact_finish(numbers + 0x7F4A7C15).view(-1) % 65536
            quantum = 2.0 ** (torch.floor(torch.log2(w.abs().clamp(min=2.0 ** -126))) - 7)
            out["w"][el] = torch.sign(w) * torch.floor(w.abs() / quantum + again.double() / 65536) * quantum
        else:
            out["w"][el] = w
        if s["master"] is not None:
            out["master"][el] = w
        if not eight:
            out["m"][el], out["v"][el] = m, v
            continue
        for name, x, bits in (("m", m, numbers % 65536), ("r", torch.sqrt(v), numbers // 65536)):
            x = x.view(-1, BLOCK)
            top = x.abs().max(1).values
            top = top * (top >= 2.0 ** -100)
            a = x.abs() * (448 / top.clamp(min=1e-300))[:, None] * (top > 0)[:, None]
            e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
            place = torch.floor(8 * (e + 6) + 8 * a / 2 ** e + (bits.double() + 0.5) / 65536).clamp(max=126)
            size = torch.where(place < 8, place / 512, 2 ** (torch.floor(place / 8) - 7) * (1 + place % 8 / 8))
            out[name][el] = (torch.sign(x) * size).view(-1)
            out[name + "_scale"][bl] = top / 448
    return out


def _exact_finish(h):
    """MurmurHash3's 32-bit finalizer."""
    h = h % 2 ** 32
    for shift, factor in ((16, 0x85EBCA6B), (13, 0xC2B2AE35)):
        h = h ^ (h // 2 ** shift)
        low, high = factor % 65536, factor // 65536
        h = (h * low + (h * high % 65536) * 65536) % 2 ** 32
    return h ^ (h // 65536)


def _exact_hash(seed, steps, tensor, blocks):
    one = lambda v: _exact_finish(torch.tensor([v], dtype=torch.int64, device=DEV))  # noqa: E731
    key = _exact_finish((one(steps) ^ seed))
    key = _exact_finish(key + tensor)
    key = _exact_finish(key ^ torch.arange(blocks, device=DEV))
    return _exact_finish(key[:, None] + torch.arange(BLOCK, device=DEV) * 2654435769)


def _exact_few(c, s):
    T, d, E, k, H = (c[n] for n in ("T", "d", "E", "k", "H"))
    x = s["x"].double()
    w1, w2, s1, s2 = _split_packed(s["packed"], c)

    def weight(codes, scale, e):
        if scale is None:
            return codes[e].double()
        n = codes[e].long()
        ex, fr = (n >> 3) & 15, (n & 7).double() / 8
        mag = torch.where(ex > 0, (1 + fr) * 2.0 ** (ex.double() - 7), fr * 2.0 ** -6)
        sc = 2.0 ** (scale[e].double() - 127)                 # [K / 128, rows, 4]
        return torch.where(n >= 128, -mag, mag) * sc.permute(1, 0, 2).reshape(len(n), -1).repeat_interleave(32, 1)

    logits = torch.sum(x[:, :, None] * s["w_router"].double(), 1) if T * d * E < 1 << 26 else x @ s["w_router"].double()
    order = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    p = torch.softmax(logits, 1).gather(1, order)
    gate = p / p.sum(1, keepdim=True)
    if s["mask"] is not None:
        order = torch.where(s["mask"][:, None] != 0, order, -1)
        gate = torch.where(s["mask"][:, None] != 0, gate, 0)
    y = torch.zeros(T, d, dtype=torch.float64, device=DEV)
    for e in range(E):
        tok, slot = torch.nonzero(order == e, as_tuple=True)
        if tok.numel():
            a = (x[tok] @ weight(w1, s1, e).t().contiguous()).view(-1, H // 32, 2, 32)
            h = (a[:, :, 0] / (1 + torch.exp(-a[:, :, 0])) * a[:, :, 1]).reshape(-1, H)
            y.index_add_(0, tok, gate[tok, slot][:, None] * (h @ weight(w2, s2, e).t().contiguous()))
    return dict(y=y, logits=logits, idx=order.int(), gate=gate)
