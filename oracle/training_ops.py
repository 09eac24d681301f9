"""Float64 oracle of layer norm, the gradients' norm and the AdamW step.  TEST INFRASTRUCTURE.

From their definitions (include/moe.h), in NumPy.  Shares no code with the HIP
library.
"""
from __future__ import annotations

import numpy as np


def layer_norm(x, residual, weight, bias, eps):
    """(sum, mean, rstd, y)."""
    s = x if residual is None else x + residual
    mean = s.mean(axis=1)
    rstd = 1.0 / np.sqrt(((s - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (s - mean[:, None]) * rstd[:, None] * weight
    return s, mean, rstd, y if bias is None else y + bias


def layer_norm_backward(dy, dsum, s, weight, mean, rstd):
    """(ds, dweight, dbias) of y = (s - mean) rstd weight + bias, plus dsum."""
    n = (s - mean[:, None]) * rstd[:, None]
    u = dy * weight
    ds = rstd[:, None] * (u - u.mean(axis=1, keepdims=True) - n * (u * n).mean(axis=1, keepdims=True))
    return ds if dsum is None else ds + dsum, (dy * n).sum(axis=0), dy.sum(axis=0)


def grad_norm(grads, max_norm=np.inf):
    """(norm, factor) of arrays together."""
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    if not np.isfinite(norm):
        return norm, np.nan
    return norm, max_norm / norm if norm > max_norm else 1.0


BLOCK = 128


def mix(h):
    """MurmurHash3's 32-bit finalizer of uint32 arrays."""
    h = np.asarray(h, np.uint32)
    with np.errstate(over="ignore"):
        h = (h ^ (h >> np.uint32(16))) * np.uint32(0x85EBCA6B)
        h = (h ^ (h >> np.uint32(13))) * np.uint32(0xC2B2AE35)
    return h ^ (h >> np.uint32(16))


def random_bits(seed, t, tensor, n):
    """A 32-bit number for each of n elements of a tensor at step t."""
    i = np.arange(n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        k = mix(mix(mix(np.uint32(t)) ^ np.uint32(seed)) + np.uint32(tensor))
        k = mix(k ^ (i // BLOCK).astype(np.uint32))
        return mix(k + (i % BLOCK).astype(np.uint32) * np.uint32(0x9E3779B9))


E4M3 = np.array([c / 512 if c < 8 else 2.0 ** (c // 8 - 7) * (1 + c % 8 / 8) for c in range(127)])


def decode8(codes, scales):
    """Values of E4M3 codes (uint8) times the scale of their 128 elements."""
    c = np.asarray(codes).astype(int)
    v = np.where(c & 127 == 127, np.nan, E4M3[np.minimum(c & 127, 126)]) * np.where(c >= 128, -1.0, 1.0)
    return v * np.repeat(np.asarray(scales, np.float64), BLOCK)[:len(v)]


def encode8(x, r16, root=False):
    """(codes, scales, place): place is the code with its fraction, before it is cut.  root: positive values of blocks
    that are not zero have a code of 1 at least."""
    n = len(x)
    blocks = -(-n // BLOCK)
    a = np.zeros(blocks * BLOCK)
    a[:n] = np.where(np.isfinite(x), np.abs(x), 0.0)
    amax = a.reshape(blocks, BLOCK).max(axis=1)
    amax[amax < 2.0 ** -100] = 0
    a = np.minimum(a * np.repeat(np.divide(448, amax, out=np.zeros(blocks), where=amax > 0), BLOCK), 448)[:n]
    c = np.minimum(np.searchsorted(E4M3, a, side="right") - 1, 125)
    lo, hi = E4M3[c], E4M3[c + 1]
    place = c + (a - lo) / (hi - lo) + (r16.astype(np.float64) + 0.5) / 65536
    code = np.minimum(np.floor(place), 126).astype(int)
    if root:
        code = np.maximum(code, (x > 0) & np.repeat(amax > 0, BLOCK)[:n])
    code = np.where(np.isfinite(x), code, 127) + np.where(x < 0, 128, 0)
    return code.astype(np.uint8), amax / 448, place


def adamw(w, g, m, v, t, lr, betas, eps, decay):
    """(w, m, v) after step t (the first is 1)."""
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    return w - lr * (m / (1 - betas[0] ** t) / (np.sqrt(v / (1 - betas[1] ** t)) + eps) + decay * w), m, v


def round_bf16(w, r16):
    """Stochastically rounded bfloat16 values of w, and their place: |w| in steps of its bfloat16, plus r16 / 2^16."""
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(w), 2.0 ** -126))) - 7)
    place = np.abs(w) / step + r16 / 65536
    return np.sign(w) * np.floor(place) * step, place
