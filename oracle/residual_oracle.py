"""Plain fp64 CPU oracle of the residual update between two blocks, of its gradients
and of what 8 bits keep of a tensor.

TEST INFRASTRUCTURE ONLY, like the other modules here: the product path never
imports it, and it shares no code with the kernels.  The forward is the
definition, one token and group at a time; the backward its adjoint by hand,
pinned against central differences of the forward in
tests/test_oracle_residual.py.
"""

from __future__ import annotations

import math

import numpy as np

from oracle.block_oracle import activation, sigmoid


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def _ends(lengths, B, T):
    if lengths is None:
        return [T] * B
    return [min(max(int(n), 0), T) for n in lengths]


def gate_value(p, act):
    """f(p) and f'(p)."""
    if act == "sigmoid":
        s = sigmoid(p)
        return s, s * (1.0 - s)
    return activation(p, act)


def _root(x, eps):
    return math.sqrt((x * x).sum() / x.size + eps)


def _ones(C, *ts):
    return [np.ones(C) if t is None else _f64(t) for t in ts]


def residual_forward(y, h=None, *, gate=None, act="silu", groups=1, post_norm=True, post_weight=None, alpha=None, pre_norm=True,
                     pre_weight=None, eps=1e-6, lengths=None):
    """h_out and n (None without pre_norm), zero behind the ends."""
    y, h, gate = _f64(y), _f64(h), _f64(gate)
    B, T, C = y.shape
    d = C // groups
    wp, a, wn = _ones(C, post_weight, alpha, pre_weight)
    h_out, n = np.zeros_like(y), np.zeros_like(y)
    for b, end in enumerate(_ends(lengths, B, T)):
        for t in range(end):
            z = y[b, t].copy()
            if post_norm:
                for g in range(groups):
                    part = slice(g * d, (g + 1) * d)
                    z[part] = z[part] / _root(z[part], eps)
                z = z * wp
            f = 1.0 if gate is None else gate_value(gate[b, t], act)[0]
            h_out[b, t] = a * f * z + (0.0 if h is None else h[b, t])
            n[b, t] = wn * h_out[b, t] / _root(h_out[b, t], eps)
    return h_out, n if pre_norm else None


def _norm_adjoint(x, dxhat, eps):
    """Of xhat = x / root."""
    r = _root(x, eps)
    return dxhat / r - x * (dxhat * x).sum() / (x.size * r ** 3)


def residual_backward(y, h_out, dh_out=None, dn=None, *, gate=None, act="silu", groups=1, post_norm=True, post_weight=None,
                      alpha=None, pre_norm=True, pre_weight=None, eps=1e-6, lengths=None):
    """Gradients of <dh_out, h_out> + <dn, n>; h_out is taken as given."""
    y, h_out, dh_out, dn, gate = map(_f64, (y, h_out, dh_out, dn, gate))
    B, T, C = y.shape
    d = C // groups
    wp, a, wn = _ones(C, post_weight, alpha, pre_weight)
    g = {k: np.zeros_like(y) for k in ("dy", "dgate", "dh")}
    g.update({k: np.zeros(C) for k in ("dalpha", "dpost_weight", "dpre_weight")})
    for b, end in enumerate(_ends(lengths, B, T)):
        for t in range(end):
            D = np.zeros(C) if dh_out is None else dh_out[b, t].copy()
            if pre_norm:
                x = h_out[b, t]
                g["dpre_weight"] += dn[b, t] * x / _root(x, eps)
                D = D + _norm_adjoint(x, wn * dn[b, t], eps)
            g["dh"][b, t] = D
            yhat = y[b, t].copy()
            parts = [slice(i * d, (i + 1) * d) for i in range(groups)] if post_norm else []
            for part in parts:
                yhat[part] = yhat[part] / _root(yhat[part], eps)
            z = yhat * wp if post_norm else yhat
            f, slope = (1.0, 0.0) if gate is None else gate_value(gate[b, t], act)
            g["dgate"][b, t] = D * a * z * slope
            g["dalpha"] += D * f * z
            dz = D * a * f
            if post_norm:
                g["dpost_weight"] += dz * yhat
                for part in parts:
                    g["dy"][b, t, part] = _norm_adjoint(y[b, t, part], (dz * wp)[part], eps)
            else:
                g["dy"][b, t] = dz
    return g


def eight_bits(x, block=32):
    """The values that 8 bits keep: a block of channels shares the smallest power of
    two (from 2^-126 on) of which 127 reach the largest magnitude; each value is the
    nearest multiple, ties to even.  A block that is not all finite becomes NaN."""
    x = _f64(x)
    out = np.zeros_like(x)
    for at in np.ndindex(*x.shape[:-1]):
        for c in range(0, x.shape[-1], block):
            part = x[at][c:c + block]
            if not np.isfinite(part).all():
                out[at][c:c + block] = np.nan
                continue
            e = -126
            while 127 * 2.0 ** e < np.abs(part).max():
                e += 1
            out[at][c:c + block] = np.round(part / 2.0 ** e) * 2.0 ** e
    return out
