"""Layouts of workspaces, on the CPU."""

import ctypes

import pytest

from delta_rule_recurrence_amd import falcon as fb


def up(n, to):
    return (n + to - 1) // to * to


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("D", [1, 3, 5, 8])
@pytest.mark.parametrize("T", [1, 64, 200, 1000])
def test_rows_of_the_scans_parameter_gradients_start_on_16_bytes(N, D, T):
    """A chunk's row of dA, dD and ddt_bias is written in pieces of 16 bytes; it
    holds D (N + 2) floats, which for odd D is no multiple of four."""
    p = fb.FalconScanProblem(1, T, D, N, 1, 0, 1, D, D, D, N, N)
    tokens = 64 if N <= 16 else 1024 // N
    chunks, subs = up(T, tokens) // tokens, tokens // 16 - 1
    maps, shared, sums = (2 + subs) * chunks * D * N, T * 2 * N, up(chunks * D * (1 + subs), 4)
    need = fb.load_library().falcon_scan_bwd_workspace_bytes(ctypes.byref(p))
    assert need == 4 * (maps + shared + sums + chunks * up(D * (N + 2), 4))
