"""fp64 oracle of the rotary positions.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The first 2 * len(inv_freq) values of a head are pairs (a, b): (i, i + r/2), or (2 i, 2 i + 1) when
interleaved.  Pair i at position p is the complex number a + i b multiplied by
scale * exp(i p inv_freq[i]), or by scale * exp(-i p inv_freq[i]) in the inverse form.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    if hasattr(x, "detach"):
        x = x.detach().to("cpu").double().numpy()
    return np.asarray(x, dtype=np.float64)


def rotate(x, positions, inv_freq, interleaved=False, inverse=False, scale=1.0):
    """x [T, heads, d], positions [T], inv_freq [r / 2]; returns float64 like x."""
    x, f, p = _f64(x).copy(), _f64(inv_freq), _f64(positions)
    half = len(f)
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    turn = scale * np.exp((-1j if inverse else 1j) * p[:, None] * f[None, :])
    z = (x[..., ia] + 1j * x[..., ib]) * turn[:, None, :]
    x[..., ia], x[..., ib] = z.real, z.imag
    return x
