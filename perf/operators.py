"""The operators around the routed block, as cases that can be timed and compared.

``own`` False: the plain form of each operator, elementary torch operations in
32 bits, rounded once where a result is stored.  ``own`` True: the library's
calls.  Both take the state that ``prepare`` makes, and return the same outputs.

Operators (the field ``op`` of a case):
  norm             root-mean-square norm with the residual's addition; for
                   act "mxfp8" the MXFP8 codes and scales of the rows as well
  norm_backward    its gradients
  balance          load-balance and z losses of the router with the per-expert
                   counts, and the gradient of both for the logits
  router_backward  gradients of the router's product from dense logit gradients
  decode           the experts of a few tokens with 4-bit (MXFP4) weights
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def listed():
    return [
        # one token being generated: latency is all there is
        dict(name="norm_one_token", op="norm", act="bf16", T=1, d=4096, residual=True),
        # the rows of the largest MXFP8 block, codes for its experts and bf16 rows for its router
        dict(name="norm_rows_mxfp8", op="norm", act="mxfp8", T=32768, d=2048, residual=True),
        # an odd float32 batch, first layer (no residual yet)
        dict(name="norm_odd_f32", op="norm", act="f32", T=777, d=192, residual=False),
        # training, the rows of the largest bf16 block
        dict(name="norm_bwd_bf16", op="norm_backward", act="bf16", T=16384, d=4096, residual=True),
        # training, an odd small batch
        dict(name="norm_bwd_odd", op="norm_backward", act="bf16", T=1000, d=256, residual=False),
        # the routers of the 64-expert block (a padded batch) and of a small block with few experts
        dict(name="balance_e64", op="balance", T=16384, E=64, k=8, padded=1500),
        dict(name="balance_e8", op="balance", T=1000, E=8, k=4, padded=0),
        # the router products' gradients: 64 experts at the largest width, 8 at a learned router's block
        dict(name="router_bwd_e64", op="router_backward", act="bf16", T=16384, d=4096, E=64),
        dict(name="router_bwd_e8", op="router_backward", act="bf16", T=8192, d=2048, E=8),
        # serving: one sequence, a ragged small batch (its last tokens padding), a full decode batch
        dict(name="decode_t1", op="decode", T=1, d=4096, E=64, k=8, H=1536, padded=0),
        dict(name="decode_t7", op="decode", T=7, d=2048, E=128, k=4, H=1024, padded=2),
        dict(name="decode_t64", op="decode", T=64, d=4096, E=64, k=8, H=1536, padded=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "balance", "router_backward", "decode"])
    if op in ("norm", "norm_backward"):
        act = rng.choice(["bf16", "bf16", "f32"] + (["mxfp8", "mxfp8"] if op == "norm" else []))
        unit = 128 if act == "mxfp8" else 64
        d = unit * _log(rng, 1, 8192 // unit)
        T = _log(rng, 1, min(32768, (1 << 26) // (d * (2 if act == "f32" else 1))))
        return dict(op=op, act=act, T=T, d=d, residual=rng.random() < 0.7)
    if op == "balance":
        E = _log(rng, 1, 1024)
        T = _log(rng, 1, min(32768, (1 << 23) // E))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 16)), padded=rng.choice([0, rng.randint(0, T)]))
    if op == "router_backward":
        act = rng.choice(["bf16", "bf16", "bf16", "f32"])
        d, E = 64 * _log(rng, 1, 64), _log(rng, 1, 256)
        T = _log(rng, 1, min(16384, (1 << (31 if act == "bf16" else 28)) // (d * E)))
        return dict(op=op, act=act, T=T, d=d, E=E)
    d, H = 128 * _log(rng, 1, 32), 128 * _log(rng, 1, 16)
    E = min(_log(rng, 1, 128), (3 << 27) // (d * H))
    T = _log(rng, 1, 128)
    return dict(op=op, T=T, d=d, E=E, k=rng.randint(1, min(E, 8)), H=H, padded=rng.choice([0, rng.randint(0, T // 2)]))


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
    """N(0, 1) rows in which one value in a hundred is 64 times larger, as residual streams have them."""
    x = _randn(g, c["T"], c["d"])
    big = torch.rand(c["T"], c["d"], generator=g, device=DEV) < 0.01
    return torch.where(big, x * 64, x).to(_store(c["act"]))


def _inputs_norm(c, g):
    return dict(x=_activations(c, g), residual=_randn(g, c["T"], c["d"]).to(_store(c["act"])) if c["residual"] else None,
                weight=(1 + 0.1 * _randn(g, c["d"])).to(_store(c["act"])))


def _inputs_norm_backward(c, g):
    dt = _store(c["act"])
    s = _activations(c, g)
    rstd = (s.double().square().mean(1) + EPS).rsqrt().float()
    return dict(s=s, rstd=rstd, dy=(0.01 * _randn(g, c["T"], c["d"])).to(dt),
                dsum=(0.01 * _randn(g, c["T"], c["d"])).to(dt) if c["residual"] else None,
                weight=(1 + 0.1 * _randn(g, c["d"])).to(dt))


def _inputs_balance(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    logits = _randn(g, T, E) + torch.linspace(0, -2, E, device=DEV)   # some experts are more popular
    idx = logits.topk(k, dim=1).indices.int()
    mask = None
    if c["padded"]:
        mask = torch.ones(T, dtype=torch.uint8, device=DEV)
        mask[torch.randperm(T, generator=g, device=DEV)[: c["padded"]]] = 0
        logits[mask == 0] = float("nan")   # what stands in a padded row must not matter
        idx[mask == 0] = -1
    return dict(logits=logits, idx=idx, mask=mask, dloss=torch.tensor([0.01, 0.001], device=DEV))


def _inputs_router_backward(c, g):
    dt = _store(c["act"])
    return dict(dlogits=1e-3 * _randn(g, c["T"], c["E"]), x=_randn(g, c["T"], c["d"]).to(dt),
                w_router=(0.02 * _randn(g, c["d"], c["E"])).to(dt), dx_in=(1e-4 * _randn(g, c["T"], c["d"])).to(dt))


def _quantize_mxfp4(w):
    """Codes (two to a byte, the even column in the low bits) and scale bytes of w [n, K] in blocks of 32 columns."""
    b = w.view(w.shape[0], -1, 32)
    e = torch.frexp(b.abs().amax(2)).exponent - 1 - 2
    a = torch.ldexp(b, -e[:, :, None].float()).clamp(-6, 6)
    mag = a.abs()
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
    mag = torch.round(mag / step) * step                                     # to even where it lies between
    code = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8) | ((b < 0).to(torch.uint8) << 3)
    code = code.view(w.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _inputs_decode(c, g):
    """The 4-bit weights are one buffer: codes of W1 [E, 2H, d/2] (rows: 32 gate, 32 up, ...) and W2 [E, d, H/2],
    scales [E, 2H, d/32] and [E, d, H/32]."""
    T, d, E, k, H = (c[n] for n in ("T", "d", "E", "k", "H"))
    logits = _randn(g, T, E)
    val, idx = logits.topk(k, dim=1)
    idx = idx.int()
    if c["padded"]:
        idx[T - c["padded"]:] = -1
    packed = torch.empty(E * 3 * d * H * 17 // 32, dtype=torch.uint8, device=DEV)
    w1, w2, s1, s2 = _split_weights(packed, c)
    for e in range(E):
        w1[e], s1[e] = _quantize_mxfp4(0.02 * _randn(g, 2 * H, d))
        w2[e], s2[e] = _quantize_mxfp4(0.02 * _randn(g, d, H))
    return dict(x=_randn(g, T, d).to(torch.bfloat16), idx=idx, gate=torch.softmax(val, 1), packed=packed)


def _split_weights(packed, c):
    d, E, H = c["d"], c["E"], c["H"]
    n = [E * 2 * H * d // 2, E * d * H // 2, E * 2 * H * d // 32, E * d * H // 32]
    w1, w2, s1, s2 = packed.split(n)
    return w1.view(E, 2 * H, d // 2), w2.view(E, d, H // 2), s1.view(E, 2 * H, d // 32), s2.view(E, d, H // 32)


# ----------------------------------------------------------------------------- one pass


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    t = s["x"].float()
    if s["residual"] is not None:
        t = t + s["residual"].float()
    rstd = torch.rsqrt((t * t).mean(1) + EPS)
    y = (t * rstd[:, None] * s["weight"].float()).to(dt)
    out = dict(y=y, rstd=rstd)
    if s["residual"] is not None:
        out["sum"] = t.to(dt)
    if c["act"] == "mxfp8":   # the codes are those of the stored row, so that they are what the block would make of it
        b = y.float().view(c["T"], -1, 32)
        amax = b.abs().amax(2)
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 8, -127).clamp(-127, 127)
        q = torch.ldexp(b, -e[:, :, None].float()).clamp(-448, 448)
        out["q"] = q.view(c["T"], -1).to(torch.float8_e4m3fn)
        out["q_scale"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _plain_norm_backward(s):
    t, rstd, dy = s["s"].float(), s["rstd"][:, None], s["dy"].float()
    u, n = dy * s["weight"].float(), t * rstd
    ds = rstd * (u - n * (u * n).mean(1, keepdim=True))
    if s["dsum"] is not None:
        ds = ds + s["dsum"].float()
    return dict(ds=ds.to(s["s"].dtype), dweight=(dy * n).sum(0))


def _plain_balance(s):
    c = s["case"]
    E, k, logits, idx = c["E"], c["k"], s["logits"], s["idx"]
    live = torch.ones(c["T"], dtype=torch.bool, device=logits.device) if s["mask"] is None else s["mask"] != 0
    logits = torch.where(live[:, None], logits, 0.0)
    N = live.sum().clamp(min=1).float()
    lse = torch.logsumexp(logits, 1)
    p = torch.exp(logits - lse[:, None])
    used = (live[:, None] & (idx >= 0) & (idx < E)).int()
    counts = torch.zeros(E, dtype=torch.int32, device=logits.device).scatter_add_(0, idx.clamp(0, E - 1).long().view(-1), used.view(-1))
    f = counts.float() / (N * k)
    P = torch.where(live[:, None], p, 0.0).sum(0) / N
    loss = torch.stack([E * (f * P).sum(), torch.where(live, lse * lse, 0.0).sum() / N])
    gb, gz = s["dloss"][0], s["dloss"][1]
    dl = p * (gb * E * (f - (p * f).sum(1, keepdim=True)) + 2 * gz * lse[:, None]) / N
    return dict(loss=loss, counts=counts, dlogits=torch.where(live[:, None], dl, 0.0))


def _plain_router_backward(s):
    dx = s["dx_in"].float() + s["dlogits"] @ s["w_router"].float().t()
    return dict(dx=dx.to(s["x"].dtype), dw_router=s["x"].float().t() @ s["dlogits"])


def _values_mxfp4(codes, scales):
    """float32 [..., K] from codes [..., K/2] and scale bytes [..., K/32]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    pair = torch.stack([table.repeat(16), table.repeat_interleave(16)], 1)     # byte -> its two values
    v = pair[codes.int()].view(*scales.shape, 32)
    return torch.ldexp(v, scales[..., None].float() - 127).view(*codes.shape[:-1], -1)


def _plain_decode(s):
    c = s["case"]
    T, d, E, k, H = (c[n] for n in ("T", "d", "E", "k", "H"))
    R = T * k
    w1, w2, s1, s2 = _split_weights(s["packed"], c)
    idx = s["idx"].view(-1).long()
    used = idx >= 0
    idx = idx.clamp(min=0)
    x = s["x"].float()
    silu = torch.nn.functional.silu
    if R <= E:      # the experts of each row, gathered
        a = (_values_mxfp4(w1[idx], s1[idx]) * x.repeat_interleave(k, 0)[:, None, :]).sum(2).view(R, H // 32, 2, 32)
        h = (silu(a[:, :, 0]) * a[:, :, 1]).reshape(R, H)
        ye = (_values_mxfp4(w2[idx], s2[idx]) * h[:, None, :]).sum(2)
    else:           # every expert on every token, and of that the rows that were asked for
        a = (x @ _values_mxfp4(w1, s1).view(E * 2 * H, d).t()).view(T, E, H // 32, 2, 32)
        h = (silu(a[:, :, :, 0]) * a[:, :, :, 1]).reshape(T, E, H).transpose(0, 1).contiguous()
        all_y = torch.bmm(h, _values_mxfp4(w2, s2).transpose(1, 2).contiguous())
        ye = all_y[idx, torch.arange(R, device=x.device) // k]
    gate = torch.where(used, s["gate"].view(-1), 0.0)
    return (gate[:, None] * ye).view(T, k, d).sum(1).to(torch.bfloat16)


# ----------------------------------------------------------------------------- the library's calls


def _handle(s, make):
    """The preallocated buffers that a program keeps from step to step."""
    if "handle" not in s:
        from routing_dispatch_grouped_router_amd import binding
        s["handle"] = make(binding)
    return s["handle"]


def _own_norm(s):
    c = s["case"]
    op = _handle(s, lambda B: B.Norm(B.problem(c["T"], c["d"], 1, 1, 128, c["act"]), DEV, eps=EPS, residual=c["residual"]))
    op(s["x"], s["weight"], residual=s["residual"])
    out = dict(y=op.y, rstd=op.rstd)
    if c["residual"]:
        out["sum"] = op.sum
    if c["act"] == "mxfp8":
        out["q"] = op.q.view(torch.float8_e4m3fn)
        out["q_scale"] = op.q_scale.view(torch.float8_e8m0fnu)
    return out


def _own_norm_backward(s):
    c = s["case"]
    op = _handle(s, lambda B: B.NormBackward(B.problem(c["T"], c["d"], 1, 1, 128, c["act"]), DEV))
    return op(s["dy"], s["s"], s["weight"], s["rstd"], dsum=s["dsum"])


def _own_balance(s):
    c = s["case"]
    op = _handle(s, lambda B: B.BalanceLoss(B.problem(c["T"], 64, c["E"], c["k"], 64, "f32"), DEV))
    op(s["logits"], s["idx"], mask=s["mask"])
    return dict(loss=op.loss, counts=op.counts, dlogits=op.backward(s["logits"], s["dloss"], mask=s["mask"]))


def _own_router_backward(s):
    c = s["case"]
    op = _handle(s, lambda B: B.RouterBackward(B.problem(c["T"], c["d"], c["E"], 1, 64, c["act"]), DEV))
    return op(s["dlogits"], s["x"], s["w_router"], dx_in=s["dx_in"])


def _own_decode(s):
    c = s["case"]
    op = _handle(s, lambda B: B.Decode(B.problem(c["T"], c["d"], c["E"], c["k"], c["H"], "bf16"), DEV))
    return op.experts(s["x"], s["idx"], s["gate"], s["packed"])


# ----------------------------------------------------------------------------- what a pass needs


def work(case):
    c = case
    T, b = c["T"], 4 if c.get("act") == "f32" else 2
    if c["op"] == "norm":
        n = T * c["d"]
        rows = n * b * (4 if c["residual"] else 2)      # x, y and with a residual that and the sum
        return dict(bytes=rows + c["d"] * b + 4 * T + (n * 33 // 32 if c["act"] == "mxfp8" else 0), flops=6 * n)
    if c["op"] == "norm_backward":
        n = T * c["d"]
        return dict(bytes=n * b * (4 if c["residual"] else 3) + c["d"] * (b + 4) + 4 * T, flops=10 * n)
    if c["op"] == "balance":
        n = (T - c["padded"]) * c["E"]
        return dict(bytes=4 * n + 4 * T * c["E"] + 4 * T * c["k"] + (T if c["padded"] else 0) + 4 * c["E"] + 16, flops=12 * n)
    if c["op"] == "router_backward":
        n = T * c["d"]
        return dict(bytes=3 * n * b + 4 * T * c["E"] + c["d"] * c["E"] * (b + 4), flops=4 * n * c["E"])
    live = T - c["padded"]
    used = c["E"] * (1 - (1 - c["k"] / c["E"]) ** live)   # distinct experts of evenly routed tokens
    return dict(bytes=int(used * 3 * c["d"] * c["H"] * 17 / 32) + 4 * T * c["d"] + 8 * T * c["k"],
                flops=6 * live * c["k"] * c["d"] * c["H"])


# ----------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    """What run() returns, from the definitions, in float64.  Values that are stored in fewer bits on the way to an
    8-bit output are rounded there, since the output is defined by them."""
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        t = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        rstd = 1 / torch.sqrt(torch.sum(t * t, 1) / c["d"] + EPS)
        y = t * (rstd[:, None] * s["weight"].double())
        out = dict(y=y, rstd=rstd)
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
    if c["op"] == "norm_backward":
        t, dy, w, r = s["s"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()
        inner = torch.sum(t * dy * w, 1)
        ds = r[:, None] * dy * w - (r ** 3 * inner / c["d"])[:, None] * t
        if s["dsum"] is not None:
            ds = ds + s["dsum"].double()
        return dict(ds=ds, dweight=torch.sum(t * dy * r[:, None], 0))
    if c["op"] == "balance":
        E, k, T = c["E"], c["k"], c["T"]
        rows = torch.arange(T, device=DEV) if s["mask"] is None else torch.nonzero(s["mask"]).view(-1)
        dl = torch.zeros(T, E, dtype=torch.float64, device=DEV)
        if rows.numel() == 0:
            return dict(loss=torch.zeros(2, dtype=torch.float64, device=DEV), counts=torch.zeros(E, dtype=torch.int32, device=DEV), dlogits=dl)
        l = s["logits"][rows].double()
        n = rows.numel()
        counts = torch.bincount(s["idx"][rows].view(-1).long(), minlength=E)
        f = counts.double() / (n * k)
        z = torch.exp(l - l.max(1, keepdim=True).values)
        p = z / z.sum(1, keepdim=True)
        lse = torch.log(z.sum(1)) + l.max(1).values
        gb, gz = (float(v) for v in s["dloss"].double())
        score = p @ f
        dl[rows] = (gb * E * p * (f[None] - score[:, None]) + gz * 2 * lse[:, None] * p) / n
        return dict(loss=torch.stack([E * score.mean(), (lse ** 2).mean()]), counts=counts.int(), dlogits=dl)
    if c["op"] == "router_backward":
        dl = s["dlogits"].double()
        return dict(dx=torch.addmm(s["dx_in"].double(), dl, s["w_router"].double().t().contiguous()),
                    dw_router=s["x"].double().t().contiguous() @ dl)
    w1, w2, s1, s2 = _split_weights(s["packed"], c)

    def weight(codes, scales):       # sign, exponent and fraction bits of each code
        n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
        ex, fr = (n >> 1) & 3, (n & 1).double()
        mag = torch.where(ex > 0, (1 + fr / 2) * 2.0 ** (ex.double() - 1), fr / 2)
        return torch.where(n >= 8, -mag, mag) * (2.0 ** (scales.double() - 127)).repeat_interleave(32, -1)

    y = torch.zeros(c["T"], c["d"], dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        tok, slot = torch.nonzero(s["idx"] == e, as_tuple=True)
        if tok.numel():
            a = s["x"][tok].double() @ weight(w1[e], s1[e]).t().contiguous()
            a = a.view(-1, c["H"] // 32, 2, 32)
            h = (a[:, :, 0] / (1 + torch.exp(-a[:, :, 0])) * a[:, :, 1]).reshape(-1, c["H"])
            y.index_add_(0, tok, s["gate"][tok, slot].double()[:, None] * (h @ weight(w2[e], s2[e]).t().contiguous()))
    return y
