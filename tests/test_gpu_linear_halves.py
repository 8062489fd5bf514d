"""The sum of a chunk's products in float32 linear attention."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

from block_utils import UNIT, cuda, f64
from test_gpu_linear import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk,dv", [(16, 64), (64, 64), (128, 128)])
def test_a_chunks_sum_in_two_halves(dk, dv):
    """64 products, none forgotten, from zero: the root mean square over 2 x 40 states.

    A rounding is off by UNIT / sqrt(3) of what it rounds, in the mean; the squares of partial sums grow
    like their terms.  If each product is rounded into its sum, two halves of 32 and their sum
    come to sqrt((2 x (1 + ... + 32) / 64 + 1) / 3) = 2.4 UNIT (one sum of 64 to 3.3), if four at a time are,
    to sqrt((2 x (1 + ... + 8) / 16 + 1) / 3) = 1.4 (one of 16 to 1.7)."""
    d = inputs(2, 40, 64, dk, dv, torch.float32, 820 + dk, carry=False, decay=0.0)
    _, S = fb.falcon_linear_fwd(*(cuda(d[n]) for n in ("q", "k", "v", "log_decay")))
    want = np.einsum("bhtk,bhtv->bhkv", f64(d["k"]), f64(d["v"]))
    off = np.linalg.norm(f64(S) - want) / np.linalg.norm(want) / UNIT
    print(f"{dk}x{dv}: {off:.2f} UNIT", flush=True)
    assert off <= 2.4
