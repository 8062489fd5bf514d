"""Values that are not finite, in scans of padded batches: what lies behind a
sequence's end has gradients of zero whatever the sequence holds, and nothing
from behind an end reaches the gradients that sum over tokens."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import block_oracle as ob

from block_utils import draws, f64, tolerance
from test_gpu_scan import device_args, inputs, oracle_args

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def agree(got, want, depth, what):
    """Not finite where the oracle is not, and the rest within the tolerance."""
    g = f64(got)
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(g), fine), f"{what}: not finite elsewhere than expected"
    norm = np.linalg.norm(want[fine])
    err = np.linalg.norm(g[fine] - want[fine]) / (norm if norm > 0 else 1.0)
    print(f"{what}: {err:.2e}", flush=True)
    assert err <= tolerance(got.dtype, depth), f"{what}: relative error {err:.3e}"


def poison(what, d, dS, lengths):
    """One value of sequence 1 (17 tokens) or 0 (none) that is not finite."""
    if what == "x":
        d["x"][1, 9, 3] = NAN
    elif what == "last x":
        d["x"][1, lengths[1] - 1, 3] = INF
    elif what == "dS_T":
        dS[1, 3, 2] = NAN
    elif what == "no tokens":
        d["S0"][0, 3, 2], dS[0, 5, 1] = NAN, INF


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("what", ["x", "last x", "dS_T", "no tokens"])
def test_scan_gradients(N, what):
    B, T, D, G = 4, 90, 40, 2
    lengths = [0, 17, 90, 64]
    case = (B, T, D, N, G, "f32", True, True, True, True, True, lengths, False)
    d, softplus, _, _ = inputs(case, seed=51)
    n = draws(52)
    dy, dS = n(B, T, D), n(B, D, N)
    poison(what, d, dS, lengths)
    with np.errstate(all="ignore"):
        want = ob.scan_backward(*(f64(d[k]) for k in ("x", "dt", "A", "B", "C")), f64(dy), dS_T=f64(dS),
                                **oracle_args(d, softplus, lengths))
    main, a = device_args(d, softplus, lengths, False)
    g = fb.falcon_scan_bwd(*main, dy.cuda(), dS_T=dS.cuda(), **a)
    for b, k in enumerate(lengths):
        for name in ("dx", "ddt", "dz", "dB", "dC"):
            assert (g[name][b, k:] == 0).all(), f"{name} behind the end of sequence {b}"
    for name, depth in (("dx", T + N), ("ddt", 2 * T + N), ("dB", T + D // G), ("dC", T + D // G), ("dA", 2 * T + B * T),
                        ("dD", B * T), ("ddt_bias", 2 * T + B * T), ("dz", T + N), ("dS0", T)):
        agree(g[name], want[name], depth, name)
