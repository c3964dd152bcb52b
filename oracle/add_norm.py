"""fp64 oracle of the root-mean-square norm with the residual's addition, its 8-bit form and its
reverse mode.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

h = x + residual, o = (1 + w) h / sqrt(mean(h^2) + eps) over the last axis; 8-bit: per group of
columns scale = max|o| / 448 and the value nearest to o / scale with 1 + 4 + 3 bits (ties to even,
largest finite value 448, subnormals in steps of 2^-9).
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().to("cpu").double().numpy()
    return np.asarray(x, dtype=np.float64)


def forward(x, residual, w, eps):
    x, residual, w = map(_f64, (x, residual, w))
    h = x if residual is None else x + residual
    return (1.0 + w) * h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps), h


def e4m3(x):
    """x rounded to 1 + 4 + 3 bits."""
    mag = np.maximum(np.abs(x), 2.0 ** -6)
    step = 2.0 ** (np.floor(np.log2(mag)) - 3)
    return np.clip(np.round(x / step) * step, -448.0, 448.0)


def quantise(o, group):
    """Returns (values before their scale, scales [.., C / group])."""
    o = _f64(o)
    g = o.reshape(*o.shape[:-1], -1, group)
    scale = np.abs(g).max(-1) / 448.0
    q = e4m3(g / np.where(scale > 0, scale, 1.0)[..., None])
    return q.reshape(o.shape), scale


def backward(h, w, d_o, d_h, eps):
    h, w, d_o, d_h = map(_f64, (h, w, d_o, d_h))
    r = 1.0 / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)
    n, dn = h * r, d_o * (1.0 + w)
    dx = r * (dn - n * np.mean(dn * n, axis=-1, keepdims=True))
    if d_h is not None:
        dx = dx + d_h
    return dict(dx=dx, dw=np.sum((d_o * n).reshape(-1, h.shape[-1]), axis=0))
