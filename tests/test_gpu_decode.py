"""The block for a few tokens with 4-bit weights (moe_pack_weights_decode,
moe_decode_experts, moe_decode) against its float64 oracle (marked gpu).

The oracle multiplies with the values the packed weights stand for; its error
bound follows float32 sums of K terms (K half-steps of the magnitudes) and h
stored as two bfloat16 terms (2^-8 of 2^-8 of it left out) through the block,
and y itself is rounded once (2^-8)."""
import numpy as np
import pytest
import torch

from oracle import block_ops as Q
from oracle import moe_oracle as O
from routing_dispatch_grouped_router_amd import binding as B
from routing_dispatch_grouped_router_amd.workloads import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _weights(rng, E, d, H):
    return [torch.from_numpy((0.05 * rng.standard_normal(s)).astype(np.float32)).to(torch.bfloat16)
            for s in ((E, d, H), (E, d, H), (E, H, d))]


def _setup(T, d, E, k, H, seed=0, **kw):
    rng = np.random.default_rng(seed + T + d + E + k + H)
    p = B.problem(T, d, E, k, H, "bf16", **kw)
    w = _weights(rng, E, d, H)
    packed = B.pack_weights_decode(p, *(t.to(DEV) for t in w))
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(torch.bfloat16)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    gate = rng.random((T, k)).astype(np.float32)
    return rng, p, w, packed, x, idx, gate


def _expect(y, x, idx, gate, packed, E, d, H):
    ref, err = Q.decode_experts(as_f64(x), idx, gate.astype(np.float64), *Q.decode_weights(packed.cpu().numpy(), E, d, H))
    got = as_f64(y)
    bad = ~(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * err)
    assert not bad.any(), f"{bad.sum()} values off, worst {np.max(np.abs(got - ref) - 2.0 ** -8 * np.abs(ref) - err):.3e}"


@pytest.mark.parametrize("E, d, H", [(1, 128, 128), (3, 256, 384), (2, 640, 128)])
def test_pack_is_the_formats_rounding(E, d, H):
    rng = np.random.default_rng(E)
    p = B.problem(1, d, E, 1, H, "bf16")
    w = _weights(rng, E, d, H)
    w[0][0, :32, 0] = 0                                       # a block of zeros
    w[0][0, :64, 1] *= 2.0 ** -100
    w[1][0, :64, 2] *= 2.0 ** 100
    w[2][0, :32, 3] = torch.tensor([5.0, -5.0, 0.25, 0.75] * 8)   # halfway values
    packed = B.pack_weights_decode(p, *(t.to(DEV) for t in w)).cpu().numpy()
    n = np.cumsum([E * H * d, E * d * H // 2, E * H * d // 16])
    w1, w2, s1, s2 = np.split(packed, n)
    src = np.stack([as_f64(t).swapaxes(1, 2).reshape(E, H // 32, 32, d) for t in w[:2]], axis=2).reshape(E, 2 * H, d)
    for codes, scales, v in ((w1, s1, src), (w2, s2, as_f64(w[2]).swapaxes(1, 2))):
        c, s = Q.mxfp4_quantize(v)
        assert np.array_equal(scales.reshape(s.shape), s)
        assert np.array_equal(Q.unpack_codes(codes.reshape(E, v.shape[1], -1)), c)


# one token and few (a group per routed row), rows and experts around the switch to a group per expert, more rows of
# one expert than a tile of 16, the most tokens, top-k at its limit
SHAPES = [(1, 128, 1, 1, 128), (1, 256, 8, 4, 128), (1, 4096, 4, 2, 256), (2, 384, 16, 8, 640), (4, 256, 16, 4, 256),
          (5, 256, 19, 4, 256), (3, 128, 64, 16, 128), (17, 512, 2, 1, 128), (33, 128, 4, 2, 384), (100, 256, 12, 3, 128),
          (256, 128, 20, 16, 128)]


@pytest.mark.parametrize("T, d, E, k, H", SHAPES)
def test_experts(T, d, E, k, H):
    print(f"[decode] T={T} d={d} E={E} k={k} H={H}", flush=True)
    rng, p, w, packed, x, idx, gate = _setup(T, d, E, k, H)
    dec = B.Decode(p, DEV)
    dec.ws.fill_(255)
    y = dec.experts(x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(gate).to(DEV), packed)
    first = y.clone()
    dec.experts(x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(gate).to(DEV), packed)
    torch.cuda.synchronize()
    assert torch.equal(first, y)
    _expect(y, x, idx, gate, packed, E, d, H)
    # a token's result does not depend on the tokens beside it
    one = B.Decode(B.problem(1, d, E, k, H, "bf16"), DEV)
    t = T // 2
    alone = one.experts(x[t:t + 1].to(DEV), torch.from_numpy(idx[t:t + 1].copy()).to(DEV),
                        torch.from_numpy(gate[t:t + 1].copy()).to(DEV), packed)
    assert torch.equal(alone[0], first[t])


# enough experts in use for workgroups whose waves take weight rows of their own (up: E H / 64 >= 512 and more rows than
# experts; down: the groups times d / 128 >= 512), with fewer slices than quarters, odd counts of them, and one expert
# of up to 16, 32 and more rows
@pytest.mark.parametrize("T, d, E, k, H", [(40, 128, 128, 4, 256), (40, 512, 128, 4, 128), (14, 640, 128, 10, 384),
                                           (31, 1152, 72, 3, 512), (100, 384, 200, 2, 256), (11, 1024, 65, 6, 128),
                                           (16, 4096, 20, 1, 128)])
def test_experts_waves_side_by_side(T, d, E, k, H):
    print(f"[decode wide] T={T} d={d} E={E} k={k} H={H}", flush=True)
    rng, p, w, packed, x, idx, gate = _setup(T, d, E, k, H, seed=2)
    for t in range(T):                                        # expert 3 in a slot of every token but the last
        if t < T - 1 and 3 not in idx[t]:
            idx[t, t % k] = 3
    idx[1, 0] = -1
    dec = B.Decode(p, DEV)
    dec.ws.fill_(255)
    args = [torch.from_numpy(idx).to(DEV), torch.from_numpy(gate).to(DEV), packed]
    y = dec.experts(x.to(DEV), *args).clone()
    for _ in range(3):
        assert torch.equal(dec.experts(x.to(DEV), *args), y)
    _expect(y, x, idx, np.where(idx >= 0, gate, 0).astype(np.float32), packed, E, d, H)
    one = B.Decode(B.problem(1, d, E, k, H, "bf16"), DEV)
    for t in (0, T - 1):
        alone = one.experts(x[t:t + 1].to(DEV), *(a[t:t + 1] for a in args[:2]), packed)
        assert torch.equal(alone[0], y[t])


@pytest.mark.parametrize("T, E", [(6, 40), (40, 6)])
def test_unused_slots_repeated_experts_and_nonfinite_rows(T, E):
    d, k, H = 256, 3, 128
    rng, p, w, packed, x, idx, gate = _setup(T, d, E, k, H, seed=9)
    idx[0] = -1                                               # a padded token
    gate[0] = np.nan
    idx[1, 1] = E
    idx[2, 0], idx[2, 2] = -2 ** 31, 2 ** 31 - 1
    gate[2, 0] = np.inf
    idx[3] = idx[3, 0]                                        # one expert in every slot
    idx[4:] = idx[5]                                          # one set of experts for most tokens
    xd = x.to(DEV)
    xd[0] = float("nan")
    dec = B.Decode(p, DEV)
    dec.ws.fill_(255)
    args = [torch.from_numpy(idx).to(DEV), torch.from_numpy(gate).to(DEV), packed]
    y = dec.experts(xd, *args).clone()
    assert not y[0].any()
    used = np.where((idx >= 0) & (idx < E), gate, 0).astype(np.float32)
    _expect(y, x, idx, used, packed, E, d, H)
    xd[5] = float("inf")                                      # its row alone
    z = dec.experts(xd, *args)
    rows = [i for i in range(T) if i != 5]
    assert torch.equal(z[rows], y[rows])
    # all tokens padded
    args[0].fill_(-1)
    assert not dec.experts(xd, *args).any()


@pytest.mark.parametrize("T, d, E, k, H, act, learned", [(1, 256, 64, 8, 128, "bf16", False),
                                                        (7, 256, 8, 2, 256, "bf16", True),
                                                        (30, 384, 20, 4, 128, "mxfp8", True),
                                                        (256, 128, 3, 1, 128, "bf16", False),
                                                        (9, 128, 520, 6, 128, "bf16", True)])
def test_block(T, d, E, k, H, act, learned):
    """moe_decode: routing bit for bit moe_route's, then the experts."""
    print(f"[decode block] T={T} d={d} E={E} k={k} H={H} {act} learned={learned}", flush=True)
    rng, _, w, packed, x, _, _ = _setup(T, d, E, k, H, seed=4)
    p = B.problem(T, d, E, k, H, act, logits_given=not learned)
    wr = torch.from_numpy((0.05 * rng.standard_normal((d, E))).astype(np.float32)).to(torch.bfloat16).to(DEV)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    xd = x.to(DEV)
    kw = dict(w_router=wr) if learned else dict(logits=logits)
    dec = B.Decode(p, DEV)
    dec.ws.fill_(255)
    y = dec(xd, packed, **kw)
    r = B.route(p, x=xd, **kw)
    torch.cuda.synchronize()
    assert torch.equal(dec.idx, r["idx"]) and torch.equal(dec.gate, r["gate"])
    if learned:
        assert torch.equal(dec.logits, r["logits"])
    assert np.array_equal(dec.idx.cpu().numpy(), O.select_topk(as_f64(r["logits"]), k))
    _expect(y, x, dec.idx.cpu().numpy(), dec.gate.cpu().numpy(), packed, E, d, H)
    before = y.clone()
    dec.idx = dec.gate = None                                 # kept in the workspace
    assert torch.equal(dec(xd, packed, **kw), before)
