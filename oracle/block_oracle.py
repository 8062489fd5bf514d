"""Plain fp64 CPU oracle of the operators around the recurrence: the short
causal convolution, the group norm with an activation and the selective state
space scan, with their gradients.

TEST INFRASTRUCTURE ONLY, like the other modules here: the product path never
imports it, and it shares no code with the kernels.  The forwards are the
definitions, one sequence, token, tap or group at a time; the backwards are
their adjoints by hand, pinned against central differences of the forwards in
tests/test_oracle_block.py.
"""

from __future__ import annotations

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def sigmoid(p):
    e = np.exp(-np.abs(p))
    return np.where(p >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def activation(p, name):
    """f(p) and f'(p)."""
    if name == "none":
        return p, np.ones_like(p)
    if name == "silu":
        s = sigmoid(p)
        return p * s, s + p * s * (1.0 - s)
    if name == "elu1":
        e = np.exp(np.minimum(p, 0.0))
        return np.where(p > 0, p + 1.0, e), np.where(p > 0, 1.0, e)
    raise ValueError(name)


def _ends(lengths, B, T):
    if lengths is None:
        return [T] * B
    return [min(max(int(n), 0), T) for n in lengths]


# ---- short causal convolution -------------------------------------------------

def conv_forward(x, weight, bias=None, *, act="silu", state=None, lengths=None):
    """y (zero behind the ends) and the last W - 1 rows up to each end."""
    x, weight, bias, state = _f64(x), _f64(weight), _f64(bias), _f64(state)
    B, T, C = x.shape
    W = weight.shape[1]
    y, out = np.zeros_like(x), np.zeros((B, W - 1, C))
    for b, n in enumerate(_ends(lengths, B, T)):
        rows = np.concatenate((np.zeros((W - 1, C)) if state is None else state[b], x[b, :n]))
        for t in range(n):
            p = np.zeros(C) if bias is None else bias.copy()
            for j in range(W):
                p += weight[:, j] * rows[t + j]
            y[b, t] = activation(p, act)[0]
        out[b] = rows[n:n + W - 1]
    return y, out


def conv_backward(x, weight, dy, bias=None, *, act="silu", state=None, lengths=None, dstate_out=None):
    x, weight, bias, state, dy, dso = map(_f64, (x, weight, bias, state, dy, dstate_out))
    B, T, C = x.shape
    W = weight.shape[1]
    g = {"dx": np.zeros_like(x), "dweight": np.zeros_like(weight), "dbias": np.zeros(C), "dstate": np.zeros((B, W - 1, C))}
    for b, n in enumerate(_ends(lengths, B, T)):
        rows = np.concatenate((np.zeros((W - 1, C)) if state is None else state[b], x[b, :n]))
        drows = np.zeros_like(rows)
        if dso is not None:
            drows[n:] += dso[b]
        for t in range(n):
            p = np.zeros(C) if bias is None else bias.copy()
            for j in range(W):
                p += weight[:, j] * rows[t + j]
            dp = dy[b, t] * activation(p, act)[1]
            g["dbias"] += dp
            for j in range(W):
                g["dweight"][:, j] += dp * rows[t + j]
                drows[t + j] += dp * weight[:, j]
        g["dstate"][b] = drows[:W - 1]
        g["dx"][b, :n] = drows[W - 1:]
    return g


# ---- group norm -----------------------------------------------------------------

def _by_token(t, layout, G):
    """[B, T, G, d] of "rows" [B, T, G d] or "heads" [B, G, T, d]."""
    if layout == "heads":
        return t.transpose(0, 2, 1, 3)
    return t.reshape(t.shape[0], t.shape[1], G, t.shape[2] // G)


def _laid(t, layout):
    if layout == "heads":
        return np.ascontiguousarray(t.transpose(0, 2, 1, 3))
    return t.reshape(t.shape[0], t.shape[1], -1)


def norm_forward(x, groups, weight=None, bias=None, *, center=False, act="none", eps=1e-6, scale=1.0, x_layout="rows",
                 y_layout="rows"):
    x = _by_token(_f64(x), x_layout, groups)
    B, T, G, d = x.shape
    w = np.ones((G, d)) if weight is None else _f64(weight).reshape(G, d)
    bb = np.zeros((G, d)) if bias is None else _f64(bias).reshape(G, d)
    y = np.empty_like(x)
    for idx in np.ndindex(B, T, G):
        v = x[idx] - (x[idx].mean() if center else 0.0)
        xhat = v / np.sqrt(np.mean(v * v) + eps)
        y[idx] = scale * activation(w[idx[2]] * xhat + bb[idx[2]], act)[0]
    return _laid(y, y_layout)


def norm_backward(x, groups, dy, weight=None, bias=None, *, center=False, act="none", eps=1e-6, scale=1.0, x_layout="rows",
                  y_layout="rows"):
    x, dy = _by_token(_f64(x), x_layout, groups), _by_token(_f64(dy), y_layout, groups)
    B, T, G, d = x.shape
    w = np.ones((G, d)) if weight is None else _f64(weight).reshape(G, d)
    bb = np.zeros((G, d)) if bias is None else _f64(bias).reshape(G, d)
    dx, dw, db = np.empty_like(x), np.zeros((G, d)), np.zeros((G, d))
    for idx in np.ndindex(B, T, G):
        g = idx[2]
        v = x[idx] - (x[idx].mean() if center else 0.0)
        dev = np.sqrt(np.mean(v * v) + eps)
        xhat = v / dev
        dp = scale * dy[idx] * activation(w[g] * xhat + bb[g], act)[1]
        dw[g] += dp * xhat
        db[g] += dp
        dh = dp * w[g]
        # xhat depends on v through v / dev and on dev through v . dv / (d dev)
        dv = dh / dev - v * np.dot(dh, v) / (d * dev ** 3)
        dx[idx] = dv - (dv.mean() if center else 0.0)
    return {"dx": _laid(dx, x_layout), "dweight": dw.reshape(-1), "dbias": db.reshape(-1)}


# ---- selective scan ----------------------------------------------------------------

def _step(dt, dt_bias, softplus):
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    if not softplus:
        return raw, raw, np.ones_like(raw)
    return raw, np.logaddexp(raw, 0.0), sigmoid(raw)


def scan_forward(x, dt, A, B, C, *, D=None, dt_bias=None, softplus=True, z=None, S0=None, lengths=None):
    """y (zero behind the ends) and the state at each end."""
    x, dt, A, B, C, D, dt_bias, z, S0 = map(_f64, (x, dt, A, B, C, D, dt_bias, z, S0))
    nb, T, W = x.shape
    G = B.shape[2]
    of = np.arange(W) // (W // G)
    delta = _step(dt, dt_bias, softplus)[1]
    y = np.zeros_like(x)
    S_T = np.zeros((nb, W, A.shape[1])) if S0 is None else S0.copy()
    for b, n in enumerate(_ends(lengths, nb, T)):
        S = S_T[b]
        for t in range(n):
            S = np.exp(delta[b, t, :, None] * A) * S + (delta[b, t] * x[b, t])[:, None] * B[b, t, of]
            read = np.einsum("cn,cn->c", C[b, t, of], S) + (0.0 if D is None else D * x[b, t])
            y[b, t] = read if z is None else read * activation(z[b, t], "silu")[0]
        S_T[b] = S
    return y, S_T


def scan_backward(x, dt, A, B, C, dy, *, D=None, dt_bias=None, softplus=True, z=None, S0=None, lengths=None, dS_T=None):
    x, dt, A, B, C, dy, D, dt_bias, z, S0, dS_T = map(_f64, (x, dt, A, B, C, dy, D, dt_bias, z, S0, dS_T))
    nb, T, W = x.shape
    N, G = A.shape[1], B.shape[2]
    of = np.arange(W) // (W // G)
    _, delta, slope = _step(dt, dt_bias, softplus)
    skip = np.zeros(W) if D is None else D
    g = {"dx": np.zeros_like(x), "ddt": np.zeros_like(x), "dz": np.zeros_like(x), "dA": np.zeros_like(A),
         "dB": np.zeros_like(B), "dC": np.zeros_like(C), "dD": np.zeros(W), "ddt_bias": np.zeros(W),
         "dS0": np.zeros((nb, W, N))}
    for b, n in enumerate(_ends(lengths, nb, T)):
        S = [np.zeros((W, N)) if S0 is None else S0[b]]
        for t in range(n):
            S.append(np.exp(delta[b, t, :, None] * A) * S[-1] + (delta[b, t] * x[b, t])[:, None] * B[b, t, of])
        dS = np.zeros((W, N)) if dS_T is None else dS_T[b].copy()
        for t in range(n - 1, -1, -1):
            q = dy[b, t]
            if z is not None:
                f, df = activation(z[b, t], "silu")
                read = np.einsum("cn,cn->c", C[b, t, of], S[t + 1]) + skip * x[b, t]
                g["dz"][b, t] = q * read * df
                q = q * f
            dS = dS + q[:, None] * C[b, t, of]
            np.add.at(g["dC"][b, t], of, q[:, None] * S[t + 1])
            np.add.at(g["dB"][b, t], of, dS * (delta[b, t] * x[b, t])[:, None])
            u = np.einsum("cn,cn->c", dS, B[b, t, of])
            a = np.exp(delta[b, t, :, None] * A)
            m = dS * a * S[t]
            g["dA"] += m * delta[b, t, :, None]
            ddt = ((m * A).sum(1) + u * x[b, t]) * slope[b, t]
            g["ddt"][b, t] = ddt
            g["ddt_bias"] += ddt
            g["dx"][b, t] = u * delta[b, t] + skip * q
            g["dD"] += q * x[b, t]
            dS = dS * a
        g["dS0"][b] = dS
    return g
