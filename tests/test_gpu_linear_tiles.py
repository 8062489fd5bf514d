"""Linear attention of heads cut into several tiles, of one chunk and of many, in every
width and type against the oracle: sums, the states between tiles, outputs, gradients.
How a head is cut is asserted, by the size of the states' slots."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import linear_oracle as lo

from block_utils import IO, close, cuda, f64
from test_gpu_linear import depth, inputs
from test_gpu_linear_decay_grad import check as check_decays

pytestmark = pytest.mark.gpu

SLOW = [-0.002, -0.02, -0.3, -2.0]   # what a tile leaves is read tiles later


def prepared(B, H, T, dk, dv, dtype, tiles, seed):
    """Seeded inputs, once the heads are known to be cut into ``tiles``."""
    p = fb.FalconLinearProblem(B, H, T, dk, dv, fb.DTYPES[IO[dtype]], 1, 1, 1, 1.0, H * dk, H * dk, H * dv)
    assert tiles > 1 and fb.falcon_linear_workspace_bytes(p) == B * H * tiles * dk * dv * 4
    d = inputs(B, H, T, dk, dv, IO[dtype], seed)
    d["log_decay"] = torch.tensor([SLOW[h % len(SLOW)] for h in range(H)])
    return d


def check(d, lengths, pick, what, scale=0.3):
    """Forward and gradients of the heads ``pick``."""
    B, H, T, dk = d["q"].shape
    dv = d["v"].shape[-1]
    D = {n: cuda(t) for n, t in d.items()}
    ends = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    a = dict(scale=scale, S0=D["S0"], lengths=ends)
    o, S_T = fb.falcon_linear_fwd(*(D[n] for n in ("q", "k", "v", "log_decay")), **a)
    g = fb.falcon_linear_bwd(*(D[n] for n in ("q", "k", "v", "log_decay", "dO")), dS_T=D["dS_T"], learned_decay=True, **a)
    cut = {n: f64(t[pick] if n == "log_decay" else t[:, pick]) for n, t in d.items()}
    a = dict(scale=scale, S0=cut["S0"], lengths=lengths)
    want, S_want = lo.linear_forward(*(cut[n] for n in ("q", "k", "v", "log_decay")), **a)
    close(o[:, pick], want, depth(T, dk), f"{what} o")
    close(S_T[:, pick], S_want, depth(T, dk), f"{what} S_T")
    ref = lo.linear_backward(*(cut[n] for n in ("q", "k", "v", "log_decay", "dO")), dS_T=cut["dS_T"], **a)
    for name in ("dq", "dk", "dv", "dS0"):
        close(g[name][:, pick], ref[name], depth(T, max(dk, dv)), f"{what} {name}")
    # every sequence's last tokens by themselves: what reaches them has passed all tiles
    for b, n in enumerate(lengths or [T] * B):
        if n > 0:
            close(o[b, pick, max(n - 3, 0):n], want[b, :, max(n - 3, 0):n], depth(T, dk), f"{what} last o of {b}")
            close(g["dv"][b, pick, :3], ref["dv"][b, :, :3], depth(T, max(dk, dv)), f"{what} first dv of {b}")
    check_decays(d, scale=scale, lengths=lengths, pick=pick, what=what)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
def test_tiles_of_one_chunk(dk, dv, dtype):
    d = prepared(2, 2, 600, dk, dv, dtype, 10, 400 + dk + dv)
    check(d, [600, 333], [0, 1], f"{dk}x{dv} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,T,dk,dv,tiles,chunks", [
    (1, 200, 800, 16, 32, 3, 5), (2, 48, 1000, 64, 64, 8, 2), (2, 48, 1500, 32, 64, 8, 3), (1, 100, 700, 128, 128, 2, 6),
    (1, 150, 1000, 64, 128, 3, 6), (3, 50, 900, 128, 32, 5, 3), (1, 300, 1100, 128, 16, 2, 9), (1, 12, 2500, 128, 128, 20, 2)])
def test_tiles_of_several_chunks(B, H, T, dk, dv, tiles, chunks, dtype):
    d = prepared(B, H, T, dk, dv, dtype, tiles, 500 + dk + dv)
    assert chunks > 1 and -(-T // (64 * chunks)) == tiles
    # ends inside the last tile, at a tile's end and inside a tile before it
    for lengths in ([T, 64 * chunks, 1][:B], [T - 70, 64 * chunks + 5, 0][:B]):
        check(d, lengths, [0, 1, 2, 3], f"{B}x{H}x{T} {dk}x{dv} {dtype} {lengths}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_prompt_goes_on_where_the_last_one_stopped(dtype):
    """The same tokens in one prompt of several tiles and in two, the state passed on."""
    d = prepared(1, 100, 1200, 64, 64, dtype, 7, 600)
    D = {n: cuda(t) for n, t in d.items()}
    cut = 700
    part = lambda a, b: [D[n][:, :, a:b].contiguous() for n in "qkv"]  # noqa: E731
    whole, S = fb.falcon_linear_fwd(*part(0, 1200), D["log_decay"], S0=D["S0"])
    first, S1 = fb.falcon_linear_fwd(*part(0, cut), D["log_decay"], S0=D["S0"])
    second, S2 = fb.falcon_linear_fwd(*part(cut, 1200), D["log_decay"], S0=S1)
    close(torch.cat((first, second), 2), f64(whole), 2 * depth(1200, 64), "o")
    close(S2, f64(S), 2 * depth(1200, 64), "S")
    assert np.isfinite(f64(whole)).all()
