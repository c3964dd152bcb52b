"""fp64 oracle of the decayed linear attention and its gradients, token by token.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Per document and head, with a constant log decay g <= 0:

    S_t = e^g S_{t-1} + k_t v_t^T,      y_t = scale S_t^T q_t.

q [T, H, d]; k, v [T, Hk, d] with Hk a divisor of H (head h uses k / v head h // (H / Hk)).
The gradients are the adjoint recurrence: with R_t = dL/dS_t,

    R_t = scale q_t dy_t^T + e^g R_{t+1}   (R after the last token: ds_final in place of e^g R)
    dq_t = scale S_t dy_t,   dk_t = R_t v_t,   dv_t = R_t^T k_t,   ds0 = e^g R_first.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().to("cpu").double().numpy()
    return np.asarray(x, dtype=np.float64)


def _expand(x, H):
    return np.repeat(x, H // x.shape[1], axis=1)


def forward(q, k, v, log_decay, cu_seqlens, s0=None, scale=1.0):
    """Packed documents.  Returns (y [T, H, d], s_final [N, H, d, d])."""
    q, k, v, g, s0 = map(_f64, (q, k, v, log_decay, s0))
    T, H, d = q.shape
    k, v = _expand(k, H), _expand(v, H)
    cu = [int(c) for c in np.asarray(cu_seqlens)]
    lam = np.exp(g)[:, None, None]
    y = np.zeros((T, H, v.shape[2]))
    last = np.zeros((len(cu) - 1, H, d, v.shape[2]))
    for n in range(len(cu) - 1):
        S = np.zeros(last.shape[1:]) if s0 is None else s0[n].copy()
        for t in range(cu[n], cu[n + 1]):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            y[t] = scale * np.matmul(q[t][:, None, :], S)[:, 0]
        last[n] = S
    return y, last


def backward(q, k, v, log_decay, cu_seqlens, dy, s0=None, ds_final=None, scale=1.0):
    """Returns dict dq, dk, dv (shapes of q, k, v) and ds0 [N, H, d, d]."""
    q, k, v, g, dy, s0, dsf = map(_f64, (q, k, v, log_decay, dy, s0, ds_final))
    T, H, d = q.shape
    Hk = k.shape[1]
    k, v = _expand(k, H), _expand(v, H)
    cu = [int(c) for c in np.asarray(cu_seqlens)]
    lam = np.exp(g)[:, None, None]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    ds0 = np.zeros((len(cu) - 1, H, d, d))
    for n in range(len(cu) - 1):
        S = np.zeros((H, d, d)) if s0 is None else s0[n].copy()
        for t in range(cu[n], cu[n + 1]):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * np.matmul(S, dy[t][:, :, None])[:, :, 0]
        R = np.zeros((H, d, d)) if dsf is None else dsf[n].copy()
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            R = R + scale * q[t][:, :, None] * dy[t][:, None, :]
            dk[t] = np.matmul(R, v[t][:, :, None])[:, :, 0]
            dv[t] = np.matmul(k[t][:, None, :], R)[:, 0]
            R = lam * R
        ds0[n] = R
    share = lambda x: x.reshape(T, Hk, H // Hk, d).sum(2)
    return dict(dq=dq, dk=share(dk), dv=share(dv), ds0=ds0)
