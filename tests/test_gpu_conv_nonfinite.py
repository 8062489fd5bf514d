"""Values that are not finite, in convolutions of padded batches: each spoils the
gradients that it belongs to, and none behind a sequence's end."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import block_oracle as ob

from block_utils import cuda, draws, f64
from test_gpu_scan_nonfinite import INF, NAN, agree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C", [24, 13])
@pytest.mark.parametrize("what", ["last x", "weight", "dstate_out", "state"])
def test_convolution_gradients(W, C, what):
    """Without an activation, so that one value spoils no more than the sums that
    it belongs to."""
    B, T = 4, 70
    lengths = [0, 17, 70, 32]
    n = draws(53)
    x, w, dy, state, dso = n(B, T, C), n(C, W), n(B, T, C), n(B, W - 1, C), n(B, W - 1, C)
    if what == "last x":
        x[1, 16, 5], x[2, 69, 6] = INF, NAN
    elif what == "weight":
        w[3, 0], w[4, W - 1] = INF, NAN
    elif what == "dstate_out":
        dso[0, 0, 2], dso[1, W - 2, 5] = NAN, INF
    else:
        state[0, W - 2, 3] = NAN            # a sequence without tokens
    a = dict(state=state, dstate_out=dso)
    with np.errstate(all="ignore"):
        want = ob.conv_backward(f64(x), f64(w), f64(dy), act="none", lengths=lengths, **{k: f64(v) for k, v in a.items()})
    g = fb.falcon_conv_bwd(x.cuda(), w.cuda(), dy.cuda(), activation="none", lengths=torch.tensor(lengths, dtype=torch.int32).cuda(),
                           grads={"dbias": torch.empty(C, device="cuda")}, **{k: cuda(v) for k, v in a.items()})
    for b, k in enumerate(lengths):
        assert (g["dx"][b, k:] == 0).all(), f"dx behind the end of sequence {b}"
    for name, depth in (("dx", 2 * W), ("dstate", 2 * W), ("dweight", B * T), ("dbias", B * T)):
        agree(g[name], want[name], depth, name)
