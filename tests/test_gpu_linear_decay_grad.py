"""The decays' gradient of linear attention, each head against its own size: heads that
forget at once beside heads that forget slowly, tiles of one chunk and of many."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import linear_oracle as lo

from block_utils import IO, UNIT, cuda, f64
from test_gpu_linear import inputs

pytestmark = pytest.mark.gpu

DECAYS = [-0.004, -0.1, -0.5, -1.0, -3.0, -5.0, -8.0, -12.0, -20.0, -60.0]


def spread(d, decay, scale, lengths=None):
    """Root of the sum of the squares of a head's terms, over pairs of tokens, tokens that read
    the first state, tokens that write into the last one, and the way between the two."""
    q, k, v, dO = (f64(d[n]) for n in ("q", "k", "v", "dO"))
    S0, R = f64(d["S0"]), f64(d["dS_T"])
    B, H, T, _ = q.shape
    total = np.zeros(H)
    for b in range(B):
        n = T if lengths is None else lengths[b]
        t = np.arange(n)
        gap = np.maximum(t[:, None] - t[None], 0)
        for h in range(H):
            g = decay[h]
            w = gap * np.exp(g * gap)
            total[h] += (w * (q[b, h, :n] @ k[b, h, :n].T) * (dO[b, h, :n] @ v[b, h, :n].T) * scale).__pow__(2).sum()
            if S0 is not None:
                reads = (t + 1) * np.exp(g * (t + 1)) * scale * ((q[b, h, :n] @ S0[b, h]) * dO[b, h, :n]).sum(-1)
                total[h] += (reads ** 2).sum()
            if R is not None:
                left = n - 1 - t
                total[h] += ((left * np.exp(g * left) * ((k[b, h, :n] @ R[b, h]) * v[b, h, :n]).sum(-1)) ** 2).sum()
            if S0 is not None and R is not None:
                total[h] += (n * np.exp(g * n) * (S0[b, h] * R[b, h]).sum()) ** 2
    return np.sqrt(total)


def check(d, *, scale=0.3, lengths=None, pick=None, what="", tiles=None):
    """``pick``: the heads that are compared.  A term is made by about 16 operations and sums
    over dk and dv products; the terms and their errors are of both signs and add like the
    roots of their squares' sums, partial sums exceed the result by a small factor, for which 4
    stands."""
    B, H, T, dk = d["q"].shape
    dv, es = d["v"].shape[-1], d["q"].dtype
    if tiles is not None:      # how a head is cut shows in the states' slots of the forward
        p = fb.FalconLinearProblem(B, H, T, dk, dv, fb.DTYPES[es], 1, 1, 1, scale, H * dk, H * dk, H * dv)
        assert fb.falcon_linear_workspace_bytes(p) == (B * H * tiles * dk * dv * 4 if tiles > 1 else 0)
    D = {n: cuda(t) for n, t in d.items()}
    ends = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    g = fb.falcon_linear_bwd(*(D[n] for n in ("q", "k", "v", "log_decay", "dO")), scale=scale, S0=D["S0"], dS_T=D["dS_T"],
                             lengths=ends, learned_decay=True)
    heads = list(range(H)) if pick is None else pick
    cut = {n: t if t is None else t[heads] if n == "log_decay" else t[:, heads] for n, t in d.items()}
    want = lo.linear_backward(*(f64(cut[n]) for n in ("q", "k", "v", "log_decay", "dO")), scale=scale, S0=f64(cut["S0"]),
                              dS_T=f64(cut["dS_T"]), lengths=lengths)["dlog_decay"]
    size = spread(cut, f64(cut["log_decay"]), scale, lengths)
    got = f64(g["dlog_decay"])[heads]
    err, most = np.abs(got - want), 4 * (16 + dk + dv) * UNIT * size
    for x in zip(f64(cut["log_decay"]), got, want, err, size):
        print(f"{what} log_decay {x[0]:g}: {x[1]:.6e} for {x[2]:.6e}, off by {x[3] / max(x[4], 1e-300):.1e} of the terms", flush=True)
    # below float32's normal numbers a factor is zero
    assert np.all(err <= most + 2.0 ** -126), f"{what}: {err / np.maximum(size, 1e-300)} of the terms, at most {4 * (16 + dk + dv) * UNIT:.1e}"


def heads_of(decays, B, H, T, dk, dv, dtype, seed, carry=True):
    d = inputs(B, H, T, dk, dv, IO[dtype], seed, carry=carry)
    d["log_decay"] = torch.tensor([decays[h % len(decays)] for h in range(H)])
    return d


@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 200, 256, 700])
def test_every_head_by_itself(T, dtype, carry):
    d = heads_of(DECAYS, 2, len(DECAYS), T, 32, 64, dtype, 300 + T, carry)
    check(d, what=f"{T} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,T,tiles", [(1, 400, 4096, 1), (1, 100, 1500, 6), (4, 80, 1024, 2), (3, 10, 300, None)])
def test_tiles_of_many_chunks(B, H, T, tiles, dtype):
    d = heads_of(DECAYS, B, H, T, 16, 32, dtype, 310 + H)
    check(d, pick=list(range(len(DECAYS))), tiles=tiles, what=f"{B}x{H}x{T} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [4, 130])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (128, 16), (32, 32), (64, 64), (64, 128), (128, 64), (128, 128)])
def test_widths(dk, dv, H, dtype):
    """Few heads in many tiles, many in one or two."""
    d = heads_of([-0.02, -0.7, -6.0, -15.0], 1, H, 600, dk, dv, dtype, 320 + dk + dv)
    check(d, pick=[0, 1, 2, 3], what=f"{dk}x{dv} {H} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [10, 200])
def test_padded_batches(H, dtype):
    """Ends inside a chunk, at a tile's, before the first token; rows behind them are NaN."""
    lengths, T = [700, 64, 0, 1, 333], 700
    d = heads_of(DECAYS, len(lengths), H, T, 16, 16, dtype, 330)
    for b, n in enumerate(lengths):
        for name in ("q", "k", "v", "dO"):
            d[name][b, :, n:] = float("nan")
    check(d, pick=list(range(10)), lengths=lengths, what=f"padded {H} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 64, 500])
def test_what_forgets_everything_has_no_gradient(T, dtype):
    d = heads_of([-float("inf"), -0.5], 2, 4, T, 32, 32, dtype, 340)
    D = {n: cuda(t) for n, t in d.items()}
    g = fb.falcon_linear_bwd(*(D[n] for n in ("q", "k", "v", "log_decay", "dO")), S0=D["S0"], dS_T=D["dS_T"], learned_decay=True)
    assert torch.all(g["dlog_decay"][::2] == 0) and torch.all(g["dlog_decay"][1::2] != 0)


def test_against_differences():
    """Central differences of the forward's 64-bit definition."""
    d = heads_of([-0.05, -1.0, -6.0], 1, 3, 150, 16, 16, "f32", 350)
    loss = lambda e: [((f64(d["dO"]) * o).sum((0, 2, 3)) + (f64(d["dS_T"]) * S).sum((0, 2, 3)))  # noqa: E731
                      for o, S in [lo.linear_forward(*(f64(d[n]) for n in "qkv"), f64(d["log_decay"]) + e, scale=0.3, S0=f64(d["S0"]))]][0]
    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    D = {n: cuda(t) for n, t in d.items()}
    g = fb.falcon_linear_bwd(*(D[n] for n in ("q", "k", "v", "log_decay", "dO")), scale=0.3, S0=D["S0"], dS_T=D["dS_T"], learned_decay=True)
    size = spread(d, f64(d["log_decay"]), 0.3)
    # differences: a step of 1e-5 leaves its square times the third derivative (under 150^2 of the
    # size) and the rounding of two losses (2^-52 of them, over the step)
    assert np.all(np.abs(f64(g["dlog_decay"]) - want) <= (4 * 48 * UNIT + 1e-10 * 150 ** 2) * size + 2.0 ** -52 * np.abs(loss(0.0)) / 1e-5 * 4)


@pytest.mark.parametrize("T,H", [(256, 3), (1000, 100)])
def test_results_are_the_same_every_time_and_do_not_depend_on_the_other_gradients(T, H):
    d = heads_of(DECAYS, 2, H, T, 32, 32, "bf16", 360)
    D = {n: cuda(t) for n, t in d.items()}
    a = [D[n] for n in ("q", "k", "v", "log_decay", "dO")]
    first = fb.falcon_linear_bwd(*a, S0=D["S0"], dS_T=D["dS_T"], learned_decay=True)
    plain = fb.falcon_linear_bwd(*a, S0=D["S0"], dS_T=D["dS_T"])
    again = fb.falcon_linear_bwd(*a, S0=D["S0"], dS_T=D["dS_T"], learned_decay=True)
    for n in ("dq", "dk", "dv", "dS0"):
        assert torch.equal(first[n], plain[n])
    assert torch.equal(first["dlog_decay"], again["dlog_decay"])
