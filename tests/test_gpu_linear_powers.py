"""The factors of the decays' gradient keep float32's bits however large their exponents."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

from block_utils import UNIT, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gap", [1, 2, 7, 16, 33, 63])
@pytest.mark.parametrize("wrote", [0, 37, 64])
def test_one_pair_of_tokens(wrote, gap, dtype):
    """One token writes 1 and one reads it: gap a^gap, inside a chunk or across chunks, for
    400 decays.

    A power is off by at most 5 UNIT: exp2 by two, its argument, a fraction of at most a half
    that is known to two roundings, by two, the base by one.  Inside a chunk a factor is a
    product of two of them and the gap, and enters another product: 14 UNIT.  Across chunks, of two of the writer's
    and two of the reader's and, of whole chunks between, one more, each product rounded once, and a
    sum of three such products adds as many again: 35."""
    H, T = 400, 192                      # a tile a head: all factors are the gradient's own
    k, q = torch.zeros(1, H, T, 16), torch.zeros(1, H, T, 16)
    k[:, :, wrote, 0], q[:, :, wrote + gap, 0] = 1, 1
    one = torch.zeros(1, H, T, 16)
    one[..., 0] = 1
    decay = -torch.linspace(0.01, 1.3, H)
    g = fb.falcon_linear_bwd(*(t.to(dtype).cuda() for t in (q, k, one)), decay.cuda(), one.to(dtype).cuda(), learned_decay=True)
    want = gap * np.exp(f64(decay) * gap)
    off = np.abs(f64(g["dlog_decay"]) / want - 1) / UNIT
    print(f"{wrote} {gap}: {off.max():.1f} UNIT", flush=True)
    assert np.all(off <= (14 if (wrote + gap) // 64 == wrote // 64 else 35))
