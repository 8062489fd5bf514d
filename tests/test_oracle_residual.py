"""Pins of the oracle of the residual update: worked numbers, parts left out, lengths,
8 bits and central differences."""

import numpy as np
import pytest

from oracle import residual_oracle as ro


def inputs(B=2, T=3, G=2, d=3, seed=1):
    n = np.random.default_rng(seed).standard_normal
    C = G * d
    return dict(y=n((B, T, C)), h=n((B, T, C)), gate=n((B, T, C)), post_weight=n(C), alpha=n(C), pre_weight=n(C))


def test_worked_numbers():
    # groups (3, 4) and (0, 5): roots sqrt(12.5) both; sigmoid(0) = 1/2
    y, h = np.array([3.0, 4, 0, 5]).reshape(1, 1, 4), np.array([1.0, 0, 0, 0]).reshape(1, 1, 4)
    r = 12.5 ** 0.5
    h_out, n = ro.residual_forward(y, h, gate=np.zeros((1, 1, 4)), act="sigmoid", groups=2, post_weight=[2, 2, 2, 4], alpha=[1, 1, 1, 0.5],
                                   pre_weight=[1, 1, 1, 3], eps=0.0)
    want = np.array([1 + 3 / r, 4 / r, 0, 5 / r])
    assert np.allclose(h_out.ravel(), want, rtol=1e-15)
    assert np.allclose(n.ravel(), want / np.sqrt((want ** 2).mean()) * [1, 1, 1, 3], rtol=1e-15)


def test_parts_left_out():
    d = inputs()
    h_out, n = ro.residual_forward(d["y"], d["h"], post_norm=False, pre_norm=False)
    assert np.allclose(h_out, d["y"] + d["h"], rtol=1e-15) and n is None
    h_out, _ = ro.residual_forward(d["y"], groups=1, eps=0.5)
    assert np.allclose(h_out, d["y"] / np.sqrt((d["y"] ** 2).mean(-1, keepdims=True) + 0.5), rtol=1e-15)
    a, _ = ro.residual_forward(d["y"], gate=d["gate"], act="none", groups=2)
    b, _ = ro.residual_forward(d["y"], gate=d["gate"], act="silu", groups=2)
    assert np.allclose(a / (1 + np.exp(-d["gate"])), b, rtol=1e-12)


def test_lengths():
    d = inputs()
    h_out, n = ro.residual_forward(**d, groups=2, lengths=[2, 0])
    whole, m = ro.residual_forward(**d, groups=2)
    assert np.array_equal(h_out[0, :2], whole[0, :2]) and np.array_equal(n[0, :2], m[0, :2])
    assert np.all(h_out[0, 2:] == 0) and np.all(h_out[1] == 0)


def test_eight_bits():
    x = np.zeros((1, 70))
    x[0, 0], x[0, 1], x[0, 2] = 127.0, 0.5, -1.5            # step 1: ties to even
    x[0, 32], x[0, 33] = 127.25, 1.0                        # 127 steps of 1 do not reach: step 2
    x[0, 64], x[0, 65] = 2.0 ** -130, 2.0 ** -126           # the smallest step
    k = ro.eight_bits(x)
    assert list(k[0, :3]) == [127.0, 0.0, -2.0]
    assert list(k[0, 32:34]) == [128.0, 0.0]
    assert list(k[0, 64:66]) == [0.0, 2.0 ** -126]
    x[0, 40] = np.inf
    k = ro.eight_bits(x)
    assert np.isnan(k[0, 32:64]).all() and np.isfinite(k[0, :32]).all()


@pytest.mark.parametrize("act", ["silu", "sigmoid", "none"])
@pytest.mark.parametrize("post,pre,lengths", [(True, True, None), (True, True, [1, 3]), (False, True, None), (True, False, None)])
def test_gradients_by_central_differences(act, post, pre, lengths):
    d = inputs()
    n = np.random.default_rng(9).standard_normal
    dh_out, dn = n(d["y"].shape), n(d["y"].shape)
    a = dict(act=act, groups=2, post_norm=post, pre_norm=pre, eps=1e-3, lengths=lengths)
    h_out, _ = ro.residual_forward(**d, **a)
    g = ro.residual_backward(d["y"], h_out, dh_out, dn, gate=d["gate"], post_weight=d["post_weight"], alpha=d["alpha"],
                             pre_weight=d["pre_weight"], **a)

    def loss(x):
        ho, no = ro.residual_forward(**x, **a)
        return (ho * dh_out).sum() + ((no * dn).sum() if pre else 0.0)

    step = 1e-6
    for name in d:
        grad = np.zeros_like(d[name])
        for at in np.ndindex(grad.shape):
            for sign in (1, -1):
                x = {k: t.copy() for k, t in d.items()}
                x[name][at] += sign * step
                grad[at] += sign * loss(x) / (2 * step)
        assert np.allclose(g["d" + name], grad, rtol=1e-6, atol=1e-7), name
