"""The short causal convolution on the GPU against the fp64 oracle: prompts,
single tokens, gradients, carried rows, padded batches, columns of a wider
projection."""

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import block_oracle as ob

from block_utils import IO, close, columns, cuda, draws, f64

pytestmark = pytest.mark.gpu

# (B, T, C, W, dtype, activation, bias, state, lengths, columns of a wider x)
CASES = [
    (1, 1, 8, 2, "bf16", "silu", True, False, None, False),
    (1, 1, 1, 4, "f32", "none", False, True, None, False),
    (2, 2, 5, 4, "bf16", "silu", True, True, None, False),      # fewer tokens than rows of state
    (3, 70, 40, 4, "bf16", "silu", True, False, [70, 1, 33], False),
    (3, 70, 40, 3, "f32", "silu", True, True, [0, 2, 70], False),
    (2, 129, 264, 4, "bf16", "silu", True, True, None, True),
    (1, 33, 1001, 3, "f32", "silu", True, True, [32], False),
    (4, 257, 16, 2, "f32", "none", True, False, None, True),
    (2, 65, 77, 4, "bf16", "none", False, True, [64, 65], True),
    (2, 300, 520, 4, "f32", "silu", True, False, None, False),
]


def inputs(case, seed=5):
    B, T, C, W, dtype, act, bias, state, lengths, wide = case
    io, n = IO[dtype], draws(seed)
    d = dict(x=n(B, T, C, dtype=io), weight=n(C, W, scale=W ** -0.5), bias=n(C, scale=0.2) if bias else None,
             state=n(B, W - 1, C, dtype=io) if state else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32))
    return d, dict(act=act, lengths=lengths)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_prompt(case):
    B, T, C, W, dtype, act, *_, lengths, wide = case
    d, o = inputs(case)
    want, rows = ob.conv_forward(f64(d["x"]), f64(d["weight"]), f64(d["bias"]), state=f64(d["state"]), **o)
    x = columns(d["x"]) if wide else d["x"].cuda()
    y, out = fb.falcon_conv_fwd(x, d["weight"].cuda(), cuda(d["bias"]), activation=act, state=cuda(d["state"]),
                                lengths=cuda(d["lengths"]), return_state=True)
    close(y, want, W, "y")
    assert (f64(out) == rows).all(), "the carried rows are copies"


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dy_type", ["f32", "bf16"])
def test_gradients(case, dy_type):
    B, T, C, W, dtype, act, *_, lengths, wide = case
    d, o = inputs(case)
    n = draws(6)
    dy, dso = n(B, T, C, dtype=IO[dy_type]), n(B, W - 1, C)
    want = ob.conv_backward(f64(d["x"]), f64(d["weight"]), f64(dy), f64(d["bias"]), state=f64(d["state"]),
                            dstate_out=f64(dso), **o)
    x = columns(d["x"]) if wide else d["x"].cuda()
    g = fb.falcon_conv_bwd(x, d["weight"].cuda(), dy.cuda(), cuda(d["bias"]), activation=act, state=cuda(d["state"]),
                           lengths=cuda(d["lengths"]), dstate_out=dso.cuda(),
                           grads={"dstate": torch.full((B, W - 1, C), 7.0, device="cuda")})
    close(g["dx"], want["dx"], 2 * W, "dx")
    close(g["dstate"], want["dstate"], 2 * W, "dstate")
    close(g["dweight"], want["dweight"], B * T, "dweight")
    if d["bias"] is not None:
        close(g["dbias"], want["dbias"], B * T, "dbias")
    else:
        assert g["dbias"] is None


@pytest.mark.parametrize("B,C,W,dtype,act,wide", [
    (1, 8, 4, "bf16", "silu", False), (5, 40, 3, "f32", "silu", True), (3, 7, 2, "bf16", "none", False),
    (33, 264, 4, "bf16", "silu", True), (64, 1001, 4, "f32", "none", False)])
def test_tokens_one_by_one_are_the_prompt(B, C, W, dtype, act, wide):
    """Every token from the rows the one before left; sequences that start anew
    at a token drop what was there."""
    io, n, T = IO[dtype], draws(9), 6
    x, w, b = n(B, T, C, dtype=io), n(C, W, scale=W ** -0.5), n(C, scale=0.2)
    state = n(B, W - 1, C, dtype=io)
    fresh = torch.arange(B) % 3 == 0
    start = torch.where(fresh[:, None, None], torch.zeros_like(state), state)
    want, rows = ob.conv_forward(f64(x), f64(w), f64(b), act=act, state=f64(start))
    s, w, b = state.cuda(), w.cuda(), b.cuda()
    for t in range(T):
        xt = columns(x[:, t]) if wide else x[:, t].contiguous().cuda()
        y = fb.falcon_conv_step(xt, w, s, b, activation=act, is_first=fresh.cuda() if t == 0 else None)
        close(y, want[:, t], W, f"token {t}")
    assert (f64(s) == rows).all()


def test_rows_behind_the_ends_stay_and_are_not_read():
    B, T, C, W = 3, 40, 24, 4
    n = draws(12)
    x, w = n(B, T, C), n(C, W)
    lengths = [0, 17, 40]
    for b, k in enumerate(lengths):
        x[b, k:] = float("nan")
    y = torch.full((B, T, C), 3.0, device="cuda")
    ends = torch.tensor(lengths, dtype=torch.int32).cuda()
    dy = n(B, T, C)
    for b, k in enumerate(lengths):
        dy[b, k:] = float("nan")
    _, out = fb.falcon_conv_fwd(x.cuda(), w.cuda(), lengths=ends, y=y, return_state=True)
    want, rows = ob.conv_forward(f64(x), f64(w), lengths=lengths)
    g = fb.falcon_conv_bwd(x.cuda(), w.cuda(), dy.cuda(), lengths=ends)
    ref = ob.conv_backward(f64(x), f64(w), f64(dy), lengths=lengths)
    for b, k in enumerate(lengths):
        assert (y[b, k:] == 3.0).all(), "rows behind the end were written"
        assert (g["dx"][b, k:] == 0.0).all(), "gradients behind the end are zero"
        if k:
            close(y[b, :k], want[b, :k], W, f"y of sequence {b}")
    assert (f64(out) == rows).all()
    close(g["dx"], ref["dx"], 2 * W, "dx")
    close(g["dweight"], ref["dweight"], B * T, "dweight")
    # lengths beyond the rows count as all of them, negative ones as none
    y2, _ = fb.falcon_conv_fwd(x.nan_to_num().cuda(), w.cuda(), lengths=torch.tensor([-5, 17, 99], dtype=torch.int32).cuda())
    assert (y2[0] == 0).all() and torch.equal(y2[2], y[2])


def test_no_tokens():
    w = draws(1)(8, 4).cuda()
    state = draws(2)(2, 3, 8).cuda()
    y, out = fb.falcon_conv_fwd(torch.empty(2, 0, 8, device="cuda"), w, state=state, return_state=True)
    assert y.shape == (2, 0, 8) and torch.equal(out, state)
    ds = draws(3)(2, 3, 8).cuda()
    g = fb.falcon_conv_bwd(torch.empty(2, 0, 8, device="cuda"), w, torch.empty(2, 0, 8, device="cuda"), w[:, 0].contiguous(),
                           state=state, dstate_out=ds)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all() and torch.equal(g["dstate"], ds)
    g = fb.falcon_conv_bwd(torch.empty(0, 5, 8, device="cuda"), w, torch.empty(0, 5, 8, device="cuda"), w[:, 0].contiguous())
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


def test_gradients_are_the_same_every_time():
    n = draws(20)
    x, w, b, dy = n(4, 500, 136).cuda(), n(136, 4).cuda(), n(136).cuda(), n(4, 500, 136).cuda()
    first = fb.falcon_conv_bwd(x, w, dy, b)
    for _ in range(3):
        again = fb.falcon_conv_bwd(x, w, dy, b)
        assert all(torch.equal(first[k], again[k]) for k in ("dx", "dweight", "dbias"))
