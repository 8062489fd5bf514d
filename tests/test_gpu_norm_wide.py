"""The norm of wide groups (more than one piece a lane) over more tokens than
there are workgroups, so that a thread walks over several, and with eps = 0."""

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import block_oracle as ob

from block_utils import IO, close, draws, f64

pytestmark = pytest.mark.gpu

# (tokens, groups, d, dtype, center, activation, eps, x layout, y layout)
CASES = [
    (8201, 1, 2048, "bf16", True, "silu", 1e-5, "rows", "rows"),
    (8201, 1, 4096, "f32", False, "elu1", 1e-5, "rows", "rows"),
    (8201, 1, 1501, "f32", True, "silu", 1e-5, "rows", "rows"),      # odd widths: four and eight pieces a lane
    (8201, 1, 3001, "bf16", False, "none", 1e-5, "heads", "rows"),
    (2101, 3, 1024, "bf16", True, "elu1", 0.0, "rows", "heads"),
    (700, 12, 64, "f32", False, "silu", 0.0, "heads", "rows"),
    (301, 5, 9, "bf16", True, "none", 0.0, "rows", "rows"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_the_oracle(case):
    T, G, d, dtype, center, act, eps, xl, yl = case
    n, io = draws(61), IO[dtype]
    shape = {"rows": (1, T, G * d), "heads": (1, G, T, d)}
    x, dy = n(*shape[xl], dtype=io, mean=0.3), n(*shape[yl])
    w, b = n(G * d, scale=0.3, mean=1.0), n(G * d, scale=0.3)
    a = dict(center=center, eps=eps, scale=0.5, x_layout=xl, y_layout=yl)
    y = fb.falcon_norm_fwd(x.cuda(), G, w.cuda(), b.cuda(), activation=act, **a)
    close(y, ob.norm_forward(f64(x), G, f64(w), f64(b), act=act, **a), d, "y")
    g = fb.falcon_norm_bwd(x.cuda(), G, dy.cuda(), w.cuda(), b.cuda(), activation=act, **a)
    want = ob.norm_backward(f64(x), G, f64(dy), f64(w), f64(b), act=act, **a)
    close(g["dx"], want["dx"], 2 * d, "dx")
    close(g["dweight"], want["dweight"], T, "dweight")
    close(g["dbias"], want["dbias"], T, "dbias")
