"""A value of linear attention that is not finite reaches what depends on it and nothing
else: outputs of its token and the later ones, gradients the other way round."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import linear_oracle as lo

from block_utils import IO, cuda, f64, tolerance
from test_gpu_linear import depth, inputs

pytestmark = pytest.mark.gpu

BAD = [float("inf"), -float("inf"), float("nan")]


def same(got, want, terms, what):
    """Not finite in the same places, and close in all others."""
    g = f64(got)
    assert np.array_equal(np.isfinite(g), np.isfinite(want)), f"{what}: {np.argwhere(np.isfinite(g) != np.isfinite(want))[:4].tolist()}"
    g, want = np.where(np.isfinite(g), g, 0), np.where(np.isfinite(want), want, 0)
    norm = np.linalg.norm(want)
    assert np.linalg.norm(g - want) <= tolerance(got.dtype, terms) * (norm if norm > 0 else 1.0), what


def check(d, lengths, what):
    T, (dk, dv) = d["q"].shape[2], d["S0"].shape[2:]
    D = {n: cuda(t) for n, t in d.items()}
    ends = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    host = [f64(d[n]) for n in ("q", "k", "v", "log_decay")]
    o, S_T = fb.falcon_linear_fwd(*(D[n] for n in ("q", "k", "v", "log_decay")), scale=0.3, S0=D["S0"], lengths=ends)
    g = fb.falcon_linear_bwd(*(D[n] for n in ("q", "k", "v", "log_decay", "dO")), scale=0.3, S0=D["S0"], dS_T=D["dS_T"], lengths=ends)
    with np.errstate(invalid="ignore", over="ignore"):
        want, S_want = lo.linear_forward(*host, scale=0.3, S0=f64(d["S0"]), lengths=lengths)
        ref = lo.linear_backward(*host, f64(d["dO"]), scale=0.3, S0=f64(d["S0"]), dS_T=f64(d["dS_T"]), lengths=lengths)
    same(o, want, depth(T, dk), f"{what} o")
    same(S_T, S_want, depth(T, dk), f"{what} S_T")
    for name in ("dq", "dk", "dv", "dS0"):
        same(g[name], ref[name], depth(T, max(dk, dv)), f"{what} {name}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (128, 16), (32, 64), (64, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("which", ["q", "k", "v", "dO"])
def test_one_value(which, dk, dv, dtype):
    """In the first and last rows of chunks, of blocks of 16 and 32 tokens and of a short last
    chunk, a sequence and head each; the heads without one stay as they are."""
    T, at = 300, [0, 15, 16, 31, 32, 47, 63, 64, 100, 255, 256, 270, 299]
    d = inputs(len(at) // 2 + 1, 2, T, dk, dv, IO[dtype], 700 + dk + dv)
    d["log_decay"] = torch.tensor([-0.01, -0.05])
    for i, t in enumerate(at):
        d[which][i // 2, i % 2, t, (5 * i) % d[which].shape[-1]] = BAD[i % 3]
    check(d, None, f"{which} {dk}x{dv} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("B,H,T", [(1, 2, 1000), (1, 110, 800), (110, 4, 300)])
def test_many_tiles_chunks_and_values(B, H, T, which, dtype):
    """Tiles of one chunk, of several, and heads of one tile; several values of a chunk, and of
    several chunks one after the other."""
    d = inputs(B, H, T, 32, 32, IO[dtype], 720 + H)
    d["log_decay"] = torch.full((H,), -0.02)
    if B > 1:
        d = {n: t if t.dim() == 1 else t[:1].expand(B, *t.shape[1:]).contiguous() for n, t in d.items()}
    for t, c, bad in ((70, 3, BAD[0]), (71, 3, BAD[1]), (90, 20, BAD[2]), (200, 7, BAD[0]), (290, 31, BAD[2])):
        d[which][B - 1, 0, t, c] = bad
    few = [B - 1]
    D = {n: cuda(t) for n, t in d.items()}
    o, S_T = fb.falcon_linear_fwd(*(D[n] for n in ("q", "k", "v", "log_decay")), scale=0.3, S0=D["S0"])
    g = fb.falcon_linear_bwd(*(D[n] for n in ("q", "k", "v", "log_decay", "dO")), scale=0.3, S0=D["S0"], dS_T=D["dS_T"])
    cut = {n: f64(t[:2] if t.dim() == 1 else t[few, :2]) for n, t in d.items()}
    host = [cut[n] for n in ("q", "k", "v", "log_decay")]
    with np.errstate(invalid="ignore", over="ignore"):
        want, S_want = lo.linear_forward(*host, scale=0.3, S0=cut["S0"])
        ref = lo.linear_backward(*host, cut["dO"], scale=0.3, S0=cut["S0"], dS_T=cut["dS_T"])
    same(o[few, :2], want, depth(T, 32), "o")
    same(S_T[few, :2], S_want, depth(T, 32), "S_T")
    for name in ("dq", "dk", "dv", "dS0"):
        same(g[name][few, :2], ref[name], depth(T, 32), name)
    # and the others as without it
    clean = fb.falcon_linear_fwd(*(torch.nan_to_num(D[n], 0, 0, 0) for n in ("q", "k", "v")), D["log_decay"], scale=0.3, S0=D["S0"])
    assert torch.equal(o[:, 1:], clean[0][:, 1:]) and torch.equal(S_T[:, 1:], clean[1][:, 1:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padded_batches(dtype):
    """The last token of a sequence, and everything behind it."""
    lengths, T = [130, 64, 199, 1], 200
    d = inputs(4, 2, T, 64, 32, IO[dtype], 740)
    d["log_decay"] = torch.tensor([-0.01, -0.05])
    for b, n in enumerate(lengths):
        for name in ("q", "k", "v", "dO"):
            d[name][b, :, n:] = float("nan")
        d["v"][b, 0, n - 1, 3] = float("inf")
        d["dO"][b, 1, 0, 5] = float("nan")
    check(d, lengths, f"padded {dtype}")


def test_prompt_and_single_tokens_agree():
    d = inputs(1, 2, 100, 32, 32, torch.float32, 760)
    d["log_decay"] = torch.tensor([-0.01, -0.05])
    d["v"][0, 0, 40, 2], d["k"][0, 1, 70, 3] = float("inf"), float("nan")
    D = {n: cuda(t) for n, t in d.items()}
    o, S_T = fb.falcon_linear_fwd(*(D[n] for n in ("q", "k", "v", "log_decay")), S0=D["S0"])
    S = D["S0"].clone()
    steps = [fb.falcon_linear_step(*(D[n][:, :, t].contiguous() for n in "qkv"), D["log_decay"], S) for t in range(100)]
    assert torch.equal(torch.isfinite(o), torch.isfinite(torch.stack(steps, 2))) and torch.equal(torch.isfinite(S), torch.isfinite(S_T))
