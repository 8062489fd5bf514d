"""Plain fp64 CPU oracle of linear attention with a decay for each head, and of its
gradients.

TEST INFRASTRUCTURE ONLY, like the other modules here: the product path never
imports it, and it shares no code with the kernels.  The forward is the
definition, a token at a time; the backward its adjoint, a token at a time from
the end, pinned against central differences of the forward and against the
masked form in tests/test_oracle_linear.py.
"""

from __future__ import annotations

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def _ends(lengths, B, T):
    if lengths is None:
        return [T] * B
    return [min(max(int(n), 0), T) for n in lengths]


def linear_forward(q, k, v, log_decay, *, scale=1.0, S0=None, lengths=None):
    """o (zero behind the ends) and the state at each end; q, k [B, H, T, dk],
    v [B, H, T, dv]."""
    q, k, v, log_decay, S0 = _f64(q), _f64(k), _f64(v), _f64(log_decay), _f64(S0)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    a = np.exp(log_decay)[:, None, None]
    o, S_T = np.zeros((B, H, T, dv)), np.zeros((B, H, dk, dv))
    for b, n in enumerate(_ends(lengths, B, T)):
        S = np.zeros((H, dk, dv)) if S0 is None else S0[b].copy()
        for t in range(n):
            S = a * S + k[b, :, t, :, None] * v[b, :, t, None, :]
            o[b, :, t] = scale * (S * q[b, :, t, :, None]).sum(1)
        S_T[b] = S
    return o, S_T


def linear_backward(q, k, v, log_decay, dO, *, scale=1.0, S0=None, lengths=None, dS_T=None):
    """Gradients of <dO, o> + <dS_T, S_T>."""
    q, k, v, log_decay, S0, dO, dS_T = (_f64(t) for t in (q, k, v, log_decay, S0, dO, dS_T))
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    a = np.exp(log_decay)[:, None, None]
    g = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dlog_decay": np.zeros(H),
         "dS0": np.zeros((B, H, dk, dv))}
    for b, n in enumerate(_ends(lengths, B, T)):
        S = np.zeros((H, dk, dv)) if S0 is None else S0[b].copy()
        before = []
        for t in range(n):
            before.append(S)
            S = a * S + k[b, :, t, :, None] * v[b, :, t, None, :]
        R = np.zeros((H, dk, dv)) if dS_T is None else dS_T[b].copy()
        for t in range(n - 1, -1, -1):
            g["dq"][b, :, t] = scale * (S * dO[b, :, t, None, :]).sum(2)
            R = R + scale * q[b, :, t, :, None] * dO[b, :, t, None, :]
            g["dk"][b, :, t] = (R * v[b, :, t, None, :]).sum(2)
            g["dv"][b, :, t] = (R * k[b, :, t, :, None]).sum(1)
            S = before.pop()
            g["dlog_decay"] += (a * S * R).sum((1, 2))
            R = a * R
        g["dS0"][b] = R
    return g
