"""Waits of the scan that give up: with a limit of no polls a wave that finds the
state not there yet does not wait for it, and the call's results are those of a
call whose waits all succeed."""

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

from test_gpu_scan import device_args, inputs

pytestmark = pytest.mark.gpu

# one chain of turns a channel; cut into chunks (few channels, 768 tokens or more)
CASES = [
    (3, 400, 100, 16, 1, "f32", True, True, True, True, True, None, False),
    (2, 300, 24, 8, 1, "bf16", True, True, True, True, False, [300, 131], False),
    (4, 500, 60, 64, 2, "f32", False, True, True, True, True, [500, 0, 17, 333], False),
    (1, 2000, 40, 16, 1, "bf16", True, True, True, True, True, None, False),
    (2, 1500, 24, 8, 2, "f32", True, True, True, True, True, [1500, 801], True),
    (1, 1201, 20, 32, 1, "f32", False, True, True, True, False, None, False),
    (3, 900, 12, 64, 1, "bf16", True, True, True, True, True, [0, 900, 333], False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_waits_that_give_up_change_nothing(case):
    d, softplus, lengths, wide = inputs(case)
    main, a = device_args(d, softplus, lengths, wide)
    y, S = fb.falcon_scan_fwd(*main, **a)
    assert y.isfinite().all() and S.isfinite().all()
    previous = fb.falcon_set_wait_limit(0)
    try:
        for _ in range(3):
            y0, S0 = fb.falcon_scan_fwd(*main, **a)
            torch.cuda.synchronize()
            assert torch.equal(y0, y) and torch.equal(S0, S)
        if a["S0"] is not None:
            # the state in place
            held = a["S0"].clone()
            y0, S0 = fb.falcon_scan_fwd(*main, S_T=held, **dict(a, S0=held))
            torch.cuda.synchronize()
            assert torch.equal(y0, y) and torch.equal(S0, S)
    finally:
        fb.falcon_set_wait_limit(previous)
    y1, S1 = fb.falcon_scan_fwd(*main, **a)
    assert torch.equal(y1, y) and torch.equal(S1, S)
