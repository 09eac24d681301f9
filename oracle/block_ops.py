"""Float64 oracle of the operators around the routed block.  TEST INFRASTRUCTURE.

The norm in front of the block, the router's losses, the dense gradients of
the router's product and the block for a few tokens with 4-bit weights, from
their definitions (include/moe.h), in NumPy.  Shares no code with the HIP
library.
"""
from __future__ import annotations

import numpy as np


def rmsnorm(x, residual, weight, eps):
    """(sum, rstd, y)."""
    s = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1) + eps)
    return s, rstd, s * rstd[:, None] * weight


def rmsnorm_backward(dy, dsum, s, weight, eps=None, rstd=None):
    """(ds, dweight) of y = s rstd(s) weight, plus dsum."""
    if rstd is None:
        rstd = 1.0 / np.sqrt((s * s).mean(axis=1) + eps)
    n = s * rstd[:, None]
    u = dy * weight
    ds = rstd[:, None] * (u - n * (u * n).mean(axis=1, keepdims=True))
    return ds if dsum is None else ds + dsum, (dy * n).sum(axis=0)


def _softmax(logits):
    mx = logits.max(axis=1, keepdims=True)
    none = np.isneginf(mx)
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(none, 0.0, np.exp(logits - np.where(none, 0.0, mx)))
        tot = z.sum(axis=1, keepdims=True)
        p = np.where(none, 0.0, z / np.where(tot == 0, 1.0, tot))
        lse = np.where(none, 0.0, np.where(none, 0.0, mx) + np.log(np.where(tot == 0, 1.0, tot)))
    return p, lse[:, 0]


def balance_loss(logits, idx, mask=None):
    """(loss [2], counts [E], N): rows that are not live are never looked at."""
    E, k = logits.shape[1], idx.shape[1]
    live = np.arange(len(logits)) if mask is None else np.flatnonzero(mask)
    N = len(live)
    chosen = idx[live].ravel()
    counts = np.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)
    if N == 0:
        return np.zeros(2), counts, 0
    p, lse = _softmax(logits[live])
    return np.array([E * (counts / (N * k) * p.mean(axis=0)).sum(), (lse ** 2).mean()]), counts, N


def balance_loss_backward(logits, counts, k, dloss, mask=None):
    E = logits.shape[1]
    live = np.arange(len(logits)) if mask is None else np.flatnonzero(mask)
    dl = np.zeros(logits.shape)
    N = len(live)
    if N:
        f = counts / (N * k)
        p, lse = _softmax(logits[live])
        dl[live] = p / N * (dloss[0] * E * (f - (p * f).sum(axis=1, keepdims=True)) + 2 * dloss[1] * lse[:, None])
    return dl


# ----------------------------------------------------------------------------- MXFP4 (OCP MX v1.0, E2M1)

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mxfp4_quantize(v):
    """(codes 0..15, scale bytes) of v [..., K], blocks of 32 along the last axis."""
    b = np.asarray(v, np.float64).reshape(*v.shape[:-1], -1, 32)
    amax = np.abs(b).max(axis=-1)
    with np.errstate(divide="ignore"):
        se = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))) - 2, -127)
    se = np.clip(se, -127, 127).astype(np.int64)
    a = np.minimum(np.abs(np.ldexp(b, -se[..., None])), 6.0)
    # nearest value of the table; halfway goes to the even code
    dist = np.abs(a[..., None] - E2M1)
    code = np.argmin(dist + np.where(np.arange(8) % 2 == 1, 1e-9, 0.0), axis=-1)
    code = code + 8 * np.signbit(b)
    return code.reshape(v.shape).astype(np.uint8), (se + 127).astype(np.uint8)


def mxfp4_values(codes, scales):
    v = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    v = v.reshape(*codes.shape[:-1], -1, 32)
    return np.ldexp(v, scales.astype(np.int64)[..., None] - 127).reshape(codes.shape)


def unpack_codes(b):
    """Codes [..., K] of bytes [..., K/2]: the even element in the low four bits."""
    return np.stack([b & 15, b >> 4], axis=-1).reshape(*b.shape[:-1], -1)


def decode_weights(packed, E, d, H):
    """(w_gate [E, d, H], w_up, w_down [E, H, d]) values of a packed MXFP4 buffer (uint8)."""
    n = np.cumsum([E * 2 * H * d // 2, E * d * H // 2, E * 2 * H * d // 32])
    w1, w2, s1, s2 = np.split(np.asarray(packed), n)
    w1 = mxfp4_values(unpack_codes(w1.reshape(E, 2 * H, d // 2)), s1.reshape(E, 2 * H, d // 32))
    w2 = mxfp4_values(unpack_codes(w2.reshape(E, d, H // 2)), s2.reshape(E, d, H // 32))
    w1 = w1.reshape(E, H // 32, 2, 32, d)
    gate, up = (np.ascontiguousarray(w1[:, :, i].reshape(E, H, d).swapaxes(1, 2)) for i in (0, 1))
    return gate, up, np.ascontiguousarray(w2.swapaxes(1, 2))


def decode_experts(x, idx, gate, wg, wu, wd, u_h=2.0 ** -16):
    """(y, bound): y[t] = sum_j gate FFN(x[t]), and how far float32 sums with h
    stored to u_h of it (as two bfloat16 terms) can be from it before y itself is rounded: with u the
    float32 half-step, a sum of n products is off by at most n u times the sum
    of their magnitudes; |silu'| < 1.1."""
    u = 2.0 ** -24
    T, d = x.shape
    H = wg.shape[2]
    y, err = np.zeros((T, d)), np.zeros((T, d))
    for t in range(T):
        for j, e in enumerate(idx[t]):
            if e < 0 or e >= len(wg):
                continue
            a, b = x[t] @ wg[e], x[t] @ wu[e]
            ea, eb = (d * u * (np.abs(x[t]) @ np.abs(w[e])) for w in (wg, wu))
            sig = 1.0 / (1.0 + np.exp(-a))
            h = a * sig * b
            # expf, the division and two products: 8 half-steps
            eh = 1.1 * np.abs(b) * ea + np.abs(a * sig) * eb + 1.1 * ea * eb + (u_h + 8 * u) * np.abs(h)
            ye = h @ wd[e]
            eye = eh @ np.abs(wd[e]) + H * u * (np.abs(h) @ np.abs(wd[e]))
            y[t] += gate[t, j] * ye
            err[t] += gate[t, j] * (eye + (len(idx[t]) + 1) * u * np.abs(ye))
    return y, err
