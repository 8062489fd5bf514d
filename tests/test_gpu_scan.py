"""The selective state space scan on the GPU against the fp64 oracle: prompts,
single tokens, gradients, carried states, padded batches, groups, columns of a
wider projection."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import block_oracle as ob

from block_utils import IO, close, columns, cuda, draws, f64

pytestmark = pytest.mark.gpu

# (B, T, D, N, G, dtype, gate, skip, dt bias, softplus, state, lengths, columns)
CASES = [
    (1, 1, 1, 8, 1, "f32", False, False, False, True, False, None, False),
    (1, 1, 64, 16, 1, "bf16", True, True, True, True, True, None, False),
    (2, 5, 96, 16, 1, "bf16", True, True, True, True, False, None, False),
    (2, 37, 200, 16, 2, "bf16", True, True, True, True, True, [37, 12], False),
    (3, 64, 65, 8, 1, "f32", False, True, True, True, True, [0, 1, 64], False),
    (1, 130, 130, 32, 2, "f32", True, False, True, True, True, None, True),
    (2, 65, 48, 64, 3, "bf16", True, True, True, False, True, [65, 33], True),
    (1, 300, 70, 16, 1, "f32", True, True, False, True, False, None, False),
    (5, 17, 12, 64, 4, "f32", False, True, True, True, False, [17, 3, 16, 9, 1], True),
    (2, 257, 136, 8, 1, "bf16", True, True, True, True, True, [255, 257], False),
    (1, 520, 24, 16, 1, "f32", True, True, True, True, True, None, False),
    # few channels and many tokens: cut into chunks
    (1, 1000, 20, 16, 1, "f32", True, True, True, True, True, None, False),
    (2, 901, 40, 8, 2, "bf16", True, True, True, True, True, [900, 130], True),
    (3, 770, 12, 64, 1, "f32", False, False, True, True, False, [0, 770, 65], False),
    (1, 768, 33, 32, 3, "f32", True, True, False, True, True, None, True),
]


def inputs(case, seed=13):
    B, T, D, N, G, dtype, gate, skip, bias, softplus, state, lengths, wide = case
    io, n = IO[dtype], draws(seed)
    d = dict(x=n(B, T, D, dtype=io), dt=n(B, T, D, dtype=io) if softplus else n(B, T, D, scale=0.05, dtype=io).abs(),
             A=-(0.2 + n(D, N).abs() * 4), B=n(B, T, G, N, dtype=io), C=n(B, T, G, N, dtype=io),
             D=n(D) if skip else None, dt_bias=n(D, scale=0.5, mean=-2.0 if softplus else 0.1).abs() * (-1 if softplus else 1) if bias else None,
             z=n(B, T, D, dtype=io) if gate else None, S0=n(B, D, N) if state else None)
    return d, softplus, lengths, wide


def oracle_args(d, softplus, lengths):
    return dict(D=f64(d["D"]), dt_bias=f64(d["dt_bias"]), softplus=softplus, z=f64(d["z"]), S0=f64(d["S0"]), lengths=lengths)


def device_args(d, softplus, lengths, wide):
    put = columns if wide else cuda
    main = [put(d["x"]), put(d["dt"]), cuda(d["A"]), shared(d["B"], wide), shared(d["C"], wide)]
    return main, dict(D=cuda(d["D"]), dt_bias=cuda(d["dt_bias"]), softplus=softplus, z=None if d["z"] is None else put(d["z"]),
                      S0=cuda(d["S0"]), lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda())


def shared(t, wide):
    """[..., G, N], or the same as columns of a wider projection."""
    return columns(t.flatten(-2)).unflatten(-1, t.shape[-2:]) if wide else t.cuda()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_prompt(case):
    d, softplus, lengths, wide = inputs(case)
    want, end = ob.scan_forward(*(f64(d[k]) for k in ("x", "dt", "A", "B", "C")), **oracle_args(d, softplus, lengths))
    main, a = device_args(d, softplus, lengths, wide)
    y, S = fb.falcon_scan_fwd(*main, **a)
    close(y, want, case[1] + case[3], "y")
    close(S, end, case[1], "S_T")


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dy_type", ["f32", "bf16"])
def test_gradients(case, dy_type):
    B, T, D, N, G = case[:5]
    d, softplus, lengths, wide = inputs(case)
    n = draws(14)
    dy, dS = n(B, T, D, dtype=IO[dy_type]), n(B, D, N)
    want = ob.scan_backward(*(f64(d[k]) for k in ("x", "dt", "A", "B", "C")), f64(dy), dS_T=f64(dS),
                            **oracle_args(d, softplus, lengths))
    main, a = device_args(d, softplus, lengths, wide)
    g = fb.falcon_scan_bwd(*main, dy.cuda(), dS_T=dS.cuda(), **a)
    for name, depth in (("dx", T + N), ("ddt", 2 * T + N), ("dB", T + D // G), ("dC", T + D // G), ("dA", 2 * T + B * T),
                        ("dD", B * T), ("ddt_bias", 2 * T + B * T), ("dz", T + N), ("dS0", T)):
        absent = {"dD": d["D"], "ddt_bias": d["dt_bias"], "dz": d["z"], "dS0": d["S0"]}
        if name in absent and absent[name] is None:
            assert g[name] is None
            continue
        close(g[name], want[name], depth, name)


@pytest.mark.parametrize("B,D,N,G,dtype,gate,wide", [
    (1, 1, 8, 1, "f32", False, False), (3, 64, 16, 1, "bf16", True, False), (5, 66, 64, 3, "f32", True, True),
    (33, 200, 16, 2, "bf16", True, True), (2, 40, 32, 1, "bf16", False, False)])
def test_tokens_one_by_one_are_the_prompt(B, D, N, G, dtype, gate, wide):
    T = 5
    d, softplus, _, _ = inputs((B, T, D, N, G, dtype, gate, True, True, True, True, None, wide), seed=15)
    fresh = torch.arange(B) % 2 == 0
    start = dict(d, S0=torch.where(fresh[:, None, None], torch.zeros_like(d["S0"]), d["S0"]))
    want, end = ob.scan_forward(*(f64(d[k]) for k in ("x", "dt", "A", "B", "C")), **oracle_args(start, softplus, None))
    S = d["S0"].cuda()
    put = columns if wide else cuda
    for t in range(T):
        one = {k: d[k][:, t].contiguous() for k in ("x", "dt", "B", "C")}
        y = fb.falcon_scan_step(put(one["x"]), put(one["dt"]), d["A"].cuda(), shared(one["B"], wide), shared(one["C"], wide), S,
                                D=d["D"].cuda(), dt_bias=d["dt_bias"].cuda(), z=put(d["z"][:, t].contiguous()) if gate else None,
                                is_first=fresh.cuda() if t == 0 else None)
        close(y, want[:, t], T + N, f"token {t}")
    close(S, end, T, "S")


def test_rows_behind_the_ends_stay_and_are_not_read():
    case = (3, 40, 72, 16, 1, "f32", True, True, True, True, True, [0, 17, 40], False)
    d, softplus, lengths, _ = inputs(case)
    dy = draws(16)(3, 40, 72)
    for b, k in enumerate(lengths):
        for name in ("x", "dt", "B", "C", "z"):
            d[name][b, k:] = float("nan")
        dy[b, k:] = float("nan")
    main, a = device_args(d, softplus, lengths, False)
    y = torch.full((3, 40, 72), 3.0, device="cuda")
    _, S = fb.falcon_scan_fwd(*main, y=y, **a)
    want, end = ob.scan_forward(*(f64(d[k]) for k in ("x", "dt", "A", "B", "C")), **oracle_args(d, softplus, lengths))
    g = fb.falcon_scan_bwd(*main, dy.cuda(), **a)
    ref = ob.scan_backward(*(f64(d[k]) for k in ("x", "dt", "A", "B", "C")), f64(dy), **oracle_args(d, softplus, lengths))
    for b, k in enumerate(lengths):
        assert (y[b, k:] == 3.0).all(), "rows behind the end were written"
        for name in ("dx", "ddt", "dz", "dB", "dC"):
            assert (g[name][b, k:] == 0).all(), f"{name} behind the end is zero"
        if k:
            close(y[b, :k], want[b, :k], k + 16, f"y of sequence {b}")
    close(S, end, 40, "S_T")
    assert torch.equal(S[0].cpu(), d["S0"][0]), "a sequence without tokens keeps its state"
    for name in ("dx", "ddt", "dz", "dA", "dB", "dC", "dD", "ddt_bias", "dS0"):
        close(g[name], ref[name], 80 + 120, name)


@pytest.mark.parametrize("T", [150, 900])
def test_state_may_be_updated_in_place(T):
    case = (2, T, 100, 16, 1, "bf16", True, True, True, True, True, None, False)
    d, softplus, _, _ = inputs(case)
    main, a = device_args(d, softplus, None, False)
    y, S = fb.falcon_scan_fwd(*main, **a)
    for _ in range(3):
        a["S0"].copy_(d["S0"])
        y2, S2 = fb.falcon_scan_fwd(*main, S_T=a["S0"], **a)
        assert S2.data_ptr() == a["S0"].data_ptr()
        assert torch.equal(y, y2) and torch.equal(S, S2)


def test_prompt_in_parts_goes_on_from_its_state():
    case = (2, 200, 72, 16, 1, "f32", True, True, True, True, True, None, False)
    d, softplus, _, _ = inputs(case)
    want, end = ob.scan_forward(*(f64(d[k]) for k in ("x", "dt", "A", "B", "C")), **oracle_args(d, softplus, None))
    main, a = device_args(d, softplus, None, False)
    S, at = a.pop("S0"), 0
    for n in (1, 70, 129):
        part = [t[:, at:at + n].contiguous() if t.dim() > 2 else t for t in main]
        z = a["z"][:, at:at + n].contiguous()
        y, S = fb.falcon_scan_fwd(*part, **dict(a, z=z, S0=S))
        close(y, want[:, at:at + n], 216, f"tokens {at} on")
        at += n
    close(S, end, 200, "S_T")


def test_no_tokens_and_no_channels():
    dev = dict(device="cuda")
    A, S0 = -torch.ones(4, 8, **dev), draws(3)(2, 4, 8).cuda()
    x, bc = torch.empty(2, 0, 4, **dev), torch.empty(2, 0, 1, 8, **dev)
    y, S = fb.falcon_scan_fwd(x, x, A, bc, bc, S0=S0)
    assert y.shape == (2, 0, 4) and torch.equal(S, S0)
    dS = draws(4)(2, 4, 8).cuda()
    g = fb.falcon_scan_bwd(x, x, A, bc, bc, x, S0=S0, dS_T=dS)
    assert (g["dA"] == 0).all() and torch.equal(g["dS0"], dS)
    x, bc = torch.empty(0, 3, 4, **dev), torch.empty(0, 3, 1, 8, **dev)
    g = fb.falcon_scan_bwd(x, x, A, bc, bc, x, D=A[:, 0].contiguous())
    assert (g["dA"] == 0).all() and (g["dD"] == 0).all()
    x, bc = torch.empty(2, 3, 0, **dev), torch.ones(2, 3, 1, 8, **dev)
    g = fb.falcon_scan_bwd(x, x, torch.empty(0, 8, **dev), bc, bc, x)
    assert (g["dB"] == 0).all() and (g["dC"] == 0).all()


def test_extreme_steps():
    """Steps of zero keep the state, steps so long that the decay underflows
    replace it, and very negative ones (softplus = exp) keep their accuracy."""
    B, T, D, N = 1, 12, 64, 16
    n = draws(17)
    d = dict(x=n(B, T, D), dt=torch.zeros(B, T, D), A=-(0.5 + n(D, N).abs()), B=n(B, T, 1, N), C=n(B, T, 1, N), D=None,
             dt_bias=None, z=None, S0=n(B, D, N))
    d["dt"][:, 0:3] = -40.0
    d["dt"][:, 3:6] = 300.0
    d["dt"][:, 6:9] = -12.0
    d["dt"][:, 9:] = -200.0          # exp(-200) is below float32: no step at all
    want, end = ob.scan_forward(*(f64(d[k]) for k in ("x", "dt", "A", "B", "C")), **oracle_args(d, True, None))
    main, a = device_args(d, True, None, False)
    y, S = fb.falcon_scan_fwd(*main, **a)
    close(y, want, T + N, "y")
    close(S, end, T, "S_T")
    for t in range(3):
        close(y[:, t], want[:, t], T + N, f"token {t}")
    dy = n(B, T, D)
    ref = ob.scan_backward(*(f64(d[k]) for k in ("x", "dt", "A", "B", "C")), f64(dy), **oracle_args(d, True, None))
    g = fb.falcon_scan_bwd(*main, dy.cuda(), **a)
    for name in ("dx", "ddt", "dA", "dB", "dC", "dS0"):
        close(g[name], ref[name], 3 * T + D, name)


def test_nan_stays_in_its_channel():
    case = (1, 50, 70, 16, 1, "f32", False, True, True, True, False, None, False)
    d, softplus, _, _ = inputs(case)
    d["x"][0, 20, 65] = float("nan")
    main, a = device_args(d, softplus, None, False)
    y, S = fb.falcon_scan_fwd(*main, **a)
    bad = torch.zeros(1, 50, 70, dtype=torch.bool)
    bad[0, 20:, 65] = True
    assert torch.equal(y.cpu().isnan(), bad)
    assert torch.equal(S.cpu().isnan().any(-1)[0], torch.arange(70) == 65)


def test_gradients_are_the_same_every_time():
    case = (2, 300, 200, 16, 2, "bf16", True, True, True, True, True, [300, 211], False)
    d, softplus, lengths, _ = inputs(case)
    main, a = device_args(d, softplus, lengths, False)
    dy = draws(18)(2, 300, 200).cuda()
    first = fb.falcon_scan_bwd(*main, dy, **a)
    for _ in range(3):
        again = fb.falcon_scan_bwd(*main, dy, **a)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_a_wait_that_gives_up_poisons_what_follows():
    """With a limit of no polls some waves go on without the state they wait for:
    the call ends all the same, and what is not NaN is right: a channel's outputs
    up to the first poisoned block of 16 tokens, and its final state only if no
    block was."""
    # channels enough that the prompt is not cut: one chain of 25 blocks each
    case = (3, 400, 100, 16, 1, "f32", True, True, True, True, True, None, False)
    d, softplus, _, _ = inputs(case)
    main, a = device_args(d, softplus, None, False)
    y, S = fb.falcon_scan_fwd(*main, **a)
    previous = fb.falcon_set_wait_limit(0)
    try:
        for _ in range(3):
            y0, S0 = fb.falcon_scan_fwd(*main, **a)
            torch.cuda.synchronize()
            lost = y0.isnan()
            assert torch.equal(y0[~lost], y[~lost])
            # once lost, lost to the end
            assert torch.equal(lost, lost.cumsum(1) > 0)
            assert torch.equal(S0.isnan().all(-1), lost[:, -1]) and torch.equal(S0[~lost[:, -1]], S[~lost[:, -1]])
    finally:
        fb.falcon_set_wait_limit(previous)
    y1, S1 = fb.falcon_scan_fwd(*main, **a)
    assert torch.equal(y1, y) and torch.equal(S1, S)
