"""Pins of the oracle of linear attention with a decay for each head: worked
numbers, the masked form, limits, continuation and central differences."""

import numpy as np
import pytest

from oracle import linear_oracle as lo


def inputs(B=2, H=2, T=7, dk=3, dv=4, seed=1):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    return dict(q=n((B, H, T, dk)), k=n((B, H, T, dk)), v=n((B, H, T, dv)), log_decay=-np.abs(n(H)), S0=n((B, H, dk, dv)))


def test_worked_numbers():
    # one head of 1 x 1, a = 1/2: S = 2, then 1/2 2 + 3 = 4, then 2 + 4 = 6
    one = lambda *x: np.array(x, float).reshape(1, 1, -1, 1)  # noqa: E731
    o, S = lo.linear_forward(one(1, 2, 3), one(1, 1, 2), one(2, 3, 2), np.log([0.5]), scale=0.1)
    assert np.allclose(o.ravel(), [0.2, 0.8, 1.8], rtol=1e-15)
    assert np.allclose(S.ravel(), [6.0], rtol=1e-15)


def test_masked_form():
    d = inputs(T=9)
    o, S_T = lo.linear_forward(**d, scale=0.7)
    T = 9
    gap = np.subtract.outer(np.arange(T), np.arange(T))
    for b in range(2):
        for h in range(2):
            a = np.exp(d["log_decay"][h])
            w = np.where(gap >= 0, a ** np.maximum(gap, 0), 0.0)
            want = (d["q"][b, h] @ d["k"][b, h].T * w) @ d["v"][b, h]
            want += (a ** np.arange(1, T + 1))[:, None] * (d["q"][b, h] @ d["S0"][b, h])
            assert np.allclose(o[b, h], 0.7 * want, rtol=1e-12)
            left = (a ** (T - 1 - np.arange(T)))[:, None]
            assert np.allclose(S_T[b, h], (d["k"][b, h] * left).T @ d["v"][b, h] + a ** T * d["S0"][b, h], rtol=1e-12)


def test_decays_of_one_and_zero():
    d = inputs()
    d["log_decay"] = np.array([0.0, -np.inf])
    o, S_T = lo.linear_forward(**d)
    assert np.allclose(S_T[:, 0], d["S0"][:, 0] + np.einsum("btk,btv->bkv", d["k"][:, 0], d["v"][:, 0]), rtol=1e-12)
    assert np.allclose(o[:, 1], (d["q"][:, 1] * d["k"][:, 1]).sum(-1, keepdims=True) * d["v"][:, 1], rtol=1e-12)


def test_continuation_and_lengths():
    d = inputs(T=8)
    o, S = lo.linear_forward(**d)
    cut = lambda x, s: {n: t[:, :, s] for n, t in x.items() if n in "qkv"}  # noqa: E731
    o1, S1 = lo.linear_forward(**cut(d, slice(0, 5)), log_decay=d["log_decay"], S0=d["S0"])
    o2, S2 = lo.linear_forward(**cut(d, slice(5, 8)), log_decay=d["log_decay"], S0=S1)
    assert np.allclose(np.concatenate((o1, o2), 2), o, rtol=1e-12) and np.allclose(S2, S, rtol=1e-12)
    ol, Sl = lo.linear_forward(**d, lengths=[5, 0])
    assert np.allclose(ol[0, :, :5], o1[0]) and np.all(ol[0, :, 5:] == 0) and np.all(ol[1] == 0)
    assert np.allclose(Sl[0], S1[0]) and np.array_equal(Sl[1], d["S0"][1])


@pytest.mark.parametrize("lengths", [None, [4, 7]])
def test_gradients_by_central_differences(lengths):
    d = inputs()
    r = np.random.default_rng(9)
    dO, dS_T = r.standard_normal((2, 2, 7, 4)), r.standard_normal((2, 2, 3, 4))
    a = dict(scale=0.6, lengths=lengths)
    g = lo.linear_backward(**d, dO=dO, dS_T=dS_T, **a)

    def loss(x):
        o, S = lo.linear_forward(**x, **a)
        return (o * dO).sum() + (S * dS_T).sum()

    step = 1e-6
    for name in d:
        grad = np.zeros_like(d[name])
        for at in np.ndindex(grad.shape):
            for sign in (1, -1):
                x = {n: t.copy() for n, t in d.items()}
                x[name][at] += sign * step
                grad[at] += sign * loss(x) / (2 * step)
        assert np.allclose(g["d" + name], grad, rtol=1e-7, atol=1e-7), name
