"""States on their way through many tiles of linear attention."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

from block_utils import UNIT, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_state_through_many_tiles(dtype):
    """One that nothing is added to, through 250 tiles of a chunk each, and its adjoint back: a^T to
    the rounding of a result (1 UNIT; 2 where the last tile's reads are made from it, of two
    factors more), for 40 decays.  (A factor in float32 is off by up to 2 UNIT every time.)"""
    H, T = 2, 250 * 64 - 7
    p = fb.FalconLinearProblem(1, H, T, 16, 16, fb.DTYPES[dtype], 1, 1, 1, 1.0, 32, 32, 32)
    assert fb.falcon_linear_workspace_bytes(p) == H * 250 * 256 * 4
    z = torch.zeros(1, H, T, 16, dtype=dtype, device="cuda")
    one = torch.ones(1, H, 16, 16, device="cuda")
    worst = 0.0
    for decay in torch.linspace(1e-5, 1e-3, 20):
        g = torch.tensor([-decay, -decay * 1.37])
        want = np.exp(f64(g) * T)
        _, S = fb.falcon_linear_fwd(z, z, z, g.cuda(), S0=one)
        grads = fb.falcon_linear_bwd(z, z, z, g.cuda(), z, S0=one, dS_T=one, learned_decay=True)
        for got, exact in ((S[0, :, 0, 0], want), (grads["dS0"][0, :, 3, 5], want), (grads["dlog_decay"], want * T * 256)):
            worst = max(worst, float(np.abs(f64(got) / exact - 1).max()) / UNIT)
    print(f"{dtype}: {worst:.1f} UNIT", flush=True)
    # the gradient adds 250 tiles' n a^n <S, R>: two states rounded once each, a power of 5 UNIT and three products
    assert worst <= 10
