"""How float32 roundings add up along a sequence of linear attention that hardly forgets."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import linear_oracle as lo

from block_utils import UNIT, cuda, f64
from test_gpu_linear import inputs

pytestmark = pytest.mark.gpu


def test_a_chunks_products_are_added_to_the_state_once():
    """Exactly: 4 x 16 times 1 to a state of 2^27, whose neighbour is 16 away."""
    H = 3
    one = torch.zeros(1, H, 128, 16)
    one[..., 0] = 1
    S0 = torch.full((1, H, 16, 16), 2.0 ** 27)
    one = one.cuda()
    _, S = fb.falcon_linear_fwd(one, one, one, torch.zeros(H, device="cuda"), S0=S0.cuda())
    S0[..., 0, 0] += 128
    assert torch.equal(S.cpu(), S0)


def test_roundings_of_a_long_float32_prompt():
    """Root mean squares over 386 heads of one tile, of 16 chunks, relative to those of the results.

    A rounding is off by UNIT / sqrt(3) of what it rounds, in the mean.  The state grows like
    the root of the tokens, so half of its squares count: two roundings of it a chunk come to
    sqrt(16 x 2 / 2 / 3) = 2.3 UNIT.  A chunk's sum takes 16 steps, sqrt(16 / 2 / 3) = 1.6, and so do scores
    and reads, from which the outputs and the decays' gradient have two such parts each more:
    sqrt(2.3^2 + 3 x 1.6^2) = 3.6.  (Sixteen roundings at the state's size come to 6.5 for it alone.)"""
    B, H, T, dk = 1, 386, 1024, 16
    d = inputs(B, H, T, dk, 16, torch.float32, 800, carry=False, decay=-0.0005)
    D = {n: cuda(t) for n, t in d.items()}
    host = [f64(d[n]) for n in ("q", "k", "v", "log_decay")]
    o, S = fb.falcon_linear_fwd(*(D[n] for n in ("q", "k", "v", "log_decay")), scale=0.3)
    g = fb.falcon_linear_bwd(*(D[n] for n in ("q", "k", "v", "log_decay", "dO")), scale=0.3, learned_decay=True)
    want, S_want = lo.linear_forward(*host, scale=0.3)
    ref = lo.linear_backward(*host, f64(d["dO"]), scale=0.3)
    for name, got, exact in (("o", o, want), ("S_T", S, S_want), ("dq", g["dq"], ref["dq"]), ("dk", g["dk"], ref["dk"]),
                             ("dv", g["dv"], ref["dv"]), ("dlog_decay", g["dlog_decay"], ref["dlog_decay"])):
        off = np.linalg.norm(f64(got) - exact) / np.linalg.norm(exact) / UNIT
        print(f"{name}: {off:.2f} UNIT", flush=True)
        assert off <= 5, name
