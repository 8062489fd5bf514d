"""A convolution of more threads than one grid holds: the sequences around the
border between two launches against the same sequences by themselves, which
agree to the bit."""

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

pytestmark = pytest.mark.gpu


def test_convolution_of_more_threads_than_a_grid():
    free, _ = torch.cuda.mem_get_info()
    if free < 64 << 30:
        pytest.skip("needs 64 GiB of device memory")
    B, C, n = 65536, 65537, 9                  # a thread each channel: past 2^32; 8.6 GB a tensor
    filled = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda").uniform_(-1, 1)  # noqa: E731
    x, state = filled(B, 1, C), filled(B, 1, C)
    w, b = filled(C, 2).float(), filled(C).float()
    ends = (torch.arange(B, device="cuda") % 3 > 0).int()
    y = torch.full((B, 1, C), 5.0, dtype=torch.bfloat16, device="cuda")
    _, out = fb.falcon_conv_fwd(x, w, b, state=state, lengths=ends, y=y, return_state=True)
    for at in (0, B // 2 + 1, B - n):
        part = slice(at, at + n)
        y2 = torch.full((n, 1, C), 5.0, dtype=torch.bfloat16, device="cuda")
        aligned = lambda t: t[part].clone()  # noqa: E731
        _, out2 = fb.falcon_conv_fwd(aligned(x), w, b, state=aligned(state), lengths=aligned(ends), y=y2, return_state=True)
        assert torch.equal(y[part], y2) and torch.equal(out[part], out2)
    del x, y, state, out
    torch.cuda.empty_cache()
