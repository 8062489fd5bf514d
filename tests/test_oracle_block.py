"""Pins of the fp64 oracle of the operators around the recurrence: its
gradients against central differences of its forwards, and closed forms of the
forwards themselves."""

import numpy as np
import pytest

from oracle import block_oracle as ob
from oracle import falcon_oracle as fo

H = 1e-5
# central differences: the truncation error is O(H^2 |f'''|) and the rounding
# error O(2^-53 |L| / H) = 1e-11 |L|; with |L|, |f'''| below about 100 each,
# both stay under 1e-7 of gradients of order one
TOL = 1e-6


def differences(loss, a):
    """dloss/da by central differences, element by element."""
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + H
        hi = loss()
        a[i] = keep - H
        lo = loss()
        a[i] = keep
        g[i] = (hi - lo) / (2 * H)
    return g


def close(got, want, what):
    err = np.abs(got - want).max() if got.size else 0.0
    assert err <= TOL * max(1.0, np.abs(want).max() if want.size else 0.0), f"{what}: {err:.2e}"


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("lengths", [None, [5, 0, 2]])
def test_conv_gradients(W, act, lengths):
    r = np.random.default_rng(W)
    x, w, b = r.standard_normal((3, 5, 2)), r.standard_normal((2, W)), r.standard_normal(2)
    s, dy, ds = r.standard_normal((3, W - 1, 2)), r.standard_normal((3, 5, 2)), r.standard_normal((3, W - 1, 2))

    def loss():
        y, out = ob.conv_forward(x, w, b, act=act, state=s, lengths=lengths)
        return (dy * y).sum() + (ds * out).sum()

    g = ob.conv_backward(x, w, dy, b, act=act, state=s, lengths=lengths, dstate_out=ds)
    for name, a in (("dx", x), ("dweight", w), ("dbias", b), ("dstate", s)):
        close(g[name], differences(loss, a), name)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("act", ["none", "silu", "elu1"])
@pytest.mark.parametrize("x_layout,y_layout", [("rows", "heads"), ("heads", "rows")])
def test_norm_gradients(center, act, x_layout, y_layout):
    r = np.random.default_rng(7)
    B, T, G, d = 2, 3, 2, 5
    shape = {"rows": (B, T, G * d), "heads": (B, G, T, d)}
    x, dy = r.standard_normal(shape[x_layout]), r.standard_normal(shape[y_layout])
    w, b = 1 + 0.3 * r.standard_normal(G * d), 0.3 * r.standard_normal(G * d)
    a = dict(center=center, act=act, eps=1e-3, scale=0.7, x_layout=x_layout, y_layout=y_layout)

    def loss():
        return (dy * ob.norm_forward(x, G, w, b, **a)).sum()

    g = ob.norm_backward(x, G, dy, w, b, **a)
    for name, t in (("dx", x), ("dweight", w), ("dbias", b)):
        close(g[name], differences(loss, t), name)


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("lengths", [None, [4, 0, 1]])
def test_scan_gradients(softplus, gate, lengths):
    r = np.random.default_rng(11)
    nb, T, D, N, G = 3, 4, 4, 3, 2
    x, dt = r.standard_normal((nb, T, D)), 0.3 * r.standard_normal((nb, T, D))
    A, B, C = -np.abs(r.standard_normal((D, N))), r.standard_normal((nb, T, G, N)), r.standard_normal((nb, T, G, N))
    skip, bias, S0 = r.standard_normal(D), 0.2 * r.standard_normal(D), r.standard_normal((nb, D, N))
    z = r.standard_normal((nb, T, D)) if gate else None
    dy, dS = r.standard_normal((nb, T, D)), r.standard_normal((nb, D, N))

    def loss():
        y, S = ob.scan_forward(x, dt, A, B, C, D=skip, dt_bias=bias, softplus=softplus, z=z, S0=S0, lengths=lengths)
        return (dy * y).sum() + (dS * S).sum()

    g = ob.scan_backward(x, dt, A, B, C, dy, D=skip, dt_bias=bias, softplus=softplus, z=z, S0=S0, lengths=lengths, dS_T=dS)
    wrt = [("dx", x), ("ddt", dt), ("dA", A), ("dB", B), ("dC", C), ("dD", skip), ("ddt_bias", bias), ("dS0", S0)]
    for name, t in wrt + ([("dz", z)] if gate else []):
        close(g[name], differences(loss, t), name)


def test_conv_is_numpy_convolve():
    r = np.random.default_rng(3)
    x, w = r.standard_normal((1, 9, 1)), r.standard_normal((1, 4))
    y, out = ob.conv_forward(x, w, act="none")
    assert np.allclose(y[0, :, 0], np.convolve(x[0, :, 0], w[0, ::-1])[:9], atol=1e-14)
    assert np.array_equal(out, x[:, -3:])


def test_conv_goes_on_from_its_state():
    r = np.random.default_rng(4)
    x, w = r.standard_normal((2, 9, 3)), r.standard_normal((3, 4))
    whole, end = ob.conv_forward(x, w)
    first, s = ob.conv_forward(x[:, :2], w)
    second, s2 = ob.conv_forward(x[:, 2:], w, state=s)
    assert np.allclose(np.concatenate((first, second), 1), whole, atol=1e-15) and np.array_equal(s2, end)


def test_norm_closed_forms():
    r = np.random.default_rng(5)
    x = r.standard_normal((2, 3, 8))
    y = ob.norm_forward(x, 2, center=True, eps=0.0)
    t = y.reshape(2, 3, 2, 4)
    assert np.allclose(t.mean(-1), 0, atol=1e-15) and np.allclose((t * t).mean(-1), 1, atol=1e-14)
    # without the mean: invariant to the input's scale, and its square sums to d
    y = ob.norm_forward(x, 2, eps=0.0)
    assert np.allclose(ob.norm_forward(3 * x, 2, eps=0.0), y, atol=1e-14)
    assert np.allclose((y.reshape(2, 3, 2, 4) ** 2).sum(-1), 4, atol=1e-13)


def test_scan_of_one_decay_is_shifted_linear_attention():
    """With A = 0, delta = 1 and no skip the scan is a running sum of x B^T,
    read by C: causal linear attention."""
    r = np.random.default_rng(6)
    x, B, C = r.standard_normal((1, 6, 2)), r.standard_normal((1, 6, 1, 3)), r.standard_normal((1, 6, 1, 3))
    y, S = ob.scan_forward(x, np.ones_like(x), np.zeros((2, 3)), B, C, softplus=False)
    mask = np.tril(C[0, :, 0] @ B[0, :, 0].T)
    assert np.allclose(y[0], mask @ x[0], atol=1e-13)
    assert np.allclose(S[0], x[0].T @ B[0, :, 0], atol=1e-13)


def test_scan_matches_the_additive_recurrence_oracle():
    """Falcon-1A with lam = 0 writes eta_t phi(k_{t-1}) v_t^T and reads with
    phi(q_t): a scan with A = 0, B_t the shifted key, x_t = v_t, delta_t = eta_t
    and C_t the query."""
    r = np.random.default_rng(8)
    T, dk, dv = 7, 3, 2
    k, q, v = r.standard_normal((1, 1, T, dk)), r.standard_normal((1, 1, T, dk)), r.standard_normal((1, 1, T, dv))
    beta = r.uniform(0.2, 1.0, (1, 1, T))
    o, S = fo.falcon_forward("falcon1a", k, q, v, beta, np.zeros((1, 1, T)), eps=0.5)
    shifted = np.concatenate((np.zeros((1, dk)), k[0, 0, :-1]))
    eta = beta[0, 0] / ((shifted ** 2).sum(1) + 0.5)
    y, S2 = ob.scan_forward(v[:, 0], np.repeat(eta[None, :, None], dv, 2), np.zeros((dv, dk)), shifted[None, :, None],
                            q[0, :, :, None, :].reshape(1, T, 1, dk), softplus=False)
    assert np.allclose(y[0], o[0, 0], atol=1e-13) and np.allclose(S2[0].T, S[0, 0], atol=1e-13)
