"""The norm of values whose squares leave float32's normal numbers: large ones, and
small ones with eps = 0."""

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import block_oracle as ob

from block_utils import IO, close, draws, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("d", [5, 64, 1000, 2048])
@pytest.mark.parametrize("exponent,eps", [(66, 1e-6), (100, 1e-6), (113, 1e-6), (63.9, 0.0), (-64, 0.0), (-90, 0.0), (-115, 0.0)])
def test_squares_out_of_range(dtype, center, d, exponent, eps):
    """Group 1 of every other token is large or small, the other groups are not."""
    n, T, G = draws(71), 6, 3
    x = n(1, T, G, d, mean=0.5)
    x[:, ::2, 1] *= 2.0 ** exponent
    x = x.flatten(2).to(IO[dtype])
    w, b, dy = n(G * d, scale=0.3, mean=1.0), n(G * d, scale=0.3), n(1, T, G * d)
    a = dict(center=center, eps=eps, scale=0.5)
    y = fb.falcon_norm_fwd(x.cuda(), G, w.cuda(), b.cuda(), activation="silu", **a)
    want = ob.norm_forward(f64(x), G, f64(w), f64(b), act="silu", **a)
    close(y, want, d, "y")
    close(y[0, 0, d:2 * d], want[0, 0, d:2 * d], d, "y of the group")
    g = fb.falcon_norm_bwd(x.cuda(), G, dy.cuda(), w.cuda(), b.cuda(), activation="silu", **a)
    ref = ob.norm_backward(f64(x), G, f64(dy), f64(w), f64(b), act="silu", **a)
    close(g["dweight"], ref["dweight"], T + d, "dweight")
    for t in range(2):
        part = (0, t, slice(d, 2 * d))
        # compared at a size of about one: dx is of the size of dy over x
        size = 2.0 ** exponent if t == 0 else 1.0
        close((g["dx"][part].double() * size).float(), ref["dx"][part] * size, 2 * d, f"dx of token {t}")
