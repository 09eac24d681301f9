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
