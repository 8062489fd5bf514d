"""The group norm with an activation on the GPU against the fp64 oracle."""

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import block_oracle as ob

from block_utils import IO, close, columns, cuda, draws, f64

pytestmark = pytest.mark.gpu

# (B, T, G, d, dtype, center, activation, weight, bias, x layout, y layout, columns of a wider x)
CASES = [
    (1, 1, 1, 1, "f32", False, "none", True, True, "rows", "rows", False),
    (1, 1, 12, 64, "bf16", False, "elu1", True, True, "rows", "heads", False),
    (2, 37, 12, 64, "bf16", True, "silu", True, True, "heads", "rows", False),
    (2, 19, 3, 128, "f32", False, "silu", True, False, "rows", "heads", True),
    (3, 7, 5, 16, "bf16", True, "none", False, True, "heads", "heads", False),
    (1, 65, 7, 9, "f32", True, "elu1", True, True, "rows", "heads", False),
    (2, 11, 2, 80, "bf16", False, "none", False, False, "rows", "rows", True),
    (2, 5, 3, 33, "bf16", True, "silu", True, True, "heads", "rows", False),
    (1, 9, 40, 32, "bf16", False, "elu1", True, True, "rows", "heads", False),   # more columns than a workgroup
    (1, 6, 2, 600, "f32", True, "silu", True, True, "rows", "rows", False),
    (1, 5, 1, 1001, "bf16", False, "silu", True, True, "rows", "heads", False),
    (1, 3, 2, 2048, "f32", True, "none", True, True, "heads", "rows", False),
    (1, 3, 1, 4096, "bf16", False, "silu", True, True, "rows", "rows", False),
    (1, 700, 6, 64, "f32", False, "elu1", True, True, "rows", "heads", True),
    (300, 3, 1, 8, "f32", True, "silu", True, True, "rows", "rows", False),
]


def inputs(case, seed=3):
    B, T, G, d, dtype, center, act, weight, bias, xl, yl, wide = case
    n, io = draws(seed), IO[dtype]
    shape = {"rows": (B, T, G * d), "heads": (B, G, T, d)}
    x = n(*shape[xl], dtype=io, mean=0.5)
    w = n(G * d, scale=0.3, mean=1.0) if weight else None
    b = n(G * d, scale=0.3) if bias else None
    a = dict(center=center, eps=1e-5, scale=0.125, x_layout=xl, y_layout=yl)
    return x, w, b, a, n(*shape[yl]), act, wide


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    x, w, b, a, _, act, wide = inputs(case)
    want = ob.norm_forward(f64(x), case[2], f64(w), f64(b), act=act, **a)
    y = fb.falcon_norm_fwd(columns(x) if wide else x.cuda(), case[2], cuda(w), cuda(b), activation=act, **a)
    close(y, want, case[3], "y")


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dy_type", ["f32", "bf16"])
def test_gradients(case, dy_type):
    x, w, b, a, dy, act, wide = inputs(case)
    B, T, G, d = case[:4]
    dy = dy.to(IO[dy_type])
    want = ob.norm_backward(f64(x), G, f64(dy), f64(w), f64(b), act=act, **a)
    g = fb.falcon_norm_bwd(columns(x) if wide else x.cuda(), G, dy.cuda(), cuda(w), cuda(b), activation=act, **a)
    if d == 1 and not a["center"]:
        # one channel: xhat = sign(x) up to eps, and dx is what cancels: of the
        # size of eps / x^2 of its two terms
        scale = abs(f64(dy) * 0.125 * f64(w) / f64(x)).max()
        assert abs(f64(g["dx"]) - want["dx"]).max() <= 64 * 2.0 ** -24 * scale
    else:
        close(g["dx"], want["dx"], 2 * d, "dx")
    for name, p in (("dweight", w), ("dbias", b)):
        if p is None:
            assert g[name] is None
        else:
            close(g[name], want[name], B * T, name)


def test_gradients_of_absent_parameters_may_be_asked_for():
    case = CASES[2]
    x, _, _, a, dy, act, _ = inputs(case)
    C = case[2] * case[3]
    want = ob.norm_backward(f64(x), case[2], f64(dy), act=act, **a)
    asked = {"dweight": torch.empty(C, device="cuda"), "dbias": torch.empty(C, device="cuda")}
    g = fb.falcon_norm_bwd(x.cuda(), case[2], dy.cuda(), activation=act, grads=asked, **a)
    assert g["dweight"] is asked["dweight"]
    close(g["dweight"], want["dweight"], case[0] * case[1], "dweight")
    close(g["dbias"], want["dbias"], case[0] * case[1], "dbias")


@pytest.mark.parametrize("center", [False, True])
def test_zero_rows_and_large_values(center):
    """A zero group norms to the bias (eps keeps it finite); float32 values near
    2^60 square to 2^120, inside the type."""
    x = torch.zeros(2, 3, 32)
    x[1, 1] = torch.linspace(-1, 1, 32) * 2.0 ** 60
    b = draws(2)(32)
    y = fb.falcon_norm_fwd(x.cuda(), 2, None, b.cuda(), center=center, eps=1e-6)
    want = ob.norm_forward(f64(x), 2, None, f64(b), center=center, eps=1e-6)
    close(y, want, 16, "y")
    assert torch.equal(y[0, 0].cpu(), b)


def test_nan_stays_in_its_group():
    x = draws(4)(2, 5, 48)
    x[1, 2, 20] = float("nan")      # group 1 of 3
    y = fb.falcon_norm_fwd(x.cuda(), 3).cpu()
    bad = torch.zeros(2, 5, 48, dtype=torch.bool)
    bad[1, 2, 16:32] = True
    assert torch.equal(y.isnan(), bad)


def test_no_tokens():
    w = torch.ones(16, device="cuda")
    x = torch.empty(2, 0, 16, device="cuda")
    assert fb.falcon_norm_fwd(x, 2, w).shape == (2, 0, 16)
    g = fb.falcon_norm_bwd(x, 2, x, w, w)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


def test_gradients_are_the_same_every_time():
    n = draws(21)
    x, w, b, dy = n(3, 400, 12 * 64).cuda(), n(768).cuda(), n(768).cuda(), n(3, 400, 768).cuda()
    first = fb.falcon_norm_bwd(x, 12, dy, w, b, activation="silu")
    for _ in range(3):
        again = fb.falcon_norm_bwd(x, 12, dy, w, b, activation="silu")
        assert all(torch.equal(first[k], again[k]) for k in first)
