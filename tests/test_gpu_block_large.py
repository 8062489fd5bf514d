"""Tensors of more than 2^32 bytes or elements: the far end of a large call against
the same rows or channels by themselves, which the small calls' tests hold to the
oracle.  Every element is computed in the same order either way, so they agree to
the bit."""

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

pytestmark = pytest.mark.gpu

GIB = 1 << 30


@pytest.fixture(autouse=True)
def room():
    free, _ = torch.cuda.mem_get_info()
    if free < 64 * GIB:
        pytest.skip("needs 64 GiB of device memory")
    yield
    torch.cuda.empty_cache()


def filled(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").uniform_(-1, 1)


def test_convolution_of_a_long_row():
    T, C, n = (1 << 26) + 5, 72, 300            # 4.8e9 elements
    x, w, b = filled(1, T, C), filled(C, 4, dtype=torch.float32), filled(C, dtype=torch.float32)
    y, state = fb.falcon_conv_fwd(x, w, b, return_state=True)
    tail = x[:, -n:].contiguous()
    y2, state2 = fb.falcon_conv_fwd(tail, w, b, state=x[:, -n - 3:-n].contiguous(), return_state=True)
    assert torch.equal(y[:, -n:], y2) and torch.equal(state, state2)


def test_gradients_of_a_convolution_of_a_long_row():
    T, C, n = (1 << 25) + 3, 72, 300            # 2.4e9 elements, 9.7e9 bytes of gradients
    x, w = filled(1, T, C), filled(C, 4, dtype=torch.float32)
    dy = filled(1, T, C)
    g = fb.falcon_conv_bwd(x, w, dy)
    g2 = fb.falcon_conv_bwd(x[:, -n:].contiguous(), w, dy[:, -n:].contiguous(), state=x[:, -n - 3:-n].contiguous())
    assert torch.equal(g["dx"][:, -n:], g2["dx"])


def test_norm_of_many_tokens():
    T, C, n = (1 << 22) + 7, 1200, 50           # 5e9 elements
    x, w = filled(1, T, C), filled(C, dtype=torch.float32)
    y = fb.falcon_norm_fwd(x, 4, w, activation="silu", y_layout="heads")
    y2 = fb.falcon_norm_fwd(x[:, -n:].contiguous(), 4, w, activation="silu", y_layout="heads")
    assert torch.equal(y[:, :, -n:], y2)


def test_scan_of_many_channels():
    B, T, D, n = 3, 700, 1 << 21, 64            # 4.4e9 elements, rows of 2^21
    x, dt = filled(B, T, D), filled(B, T, D)
    A = -1 - filled(D, 16, dtype=torch.float32).abs()
    b, c = filled(B, T, 1, 16), filled(B, T, 1, 16)
    y, S = fb.falcon_scan_fwd(x, dt, A, b, c)
    far = lambda t: t[..., -n:].contiguous()  # noqa: E731
    y2, S2 = fb.falcon_scan_fwd(far(x), far(dt), A[-n:].contiguous(), b, c)
    assert torch.equal(y[..., -n:], y2) and torch.equal(S[:, -n:], S2)


def test_gradients_of_a_scan_of_many_channels():
    T, D, n = 520, 1 << 21, 64                  # 1.1e9 elements, 4.4e9 bytes of each gradient
    x, dt, dy = filled(1, T, D), filled(1, T, D), filled(1, T, D)
    A = -1 - filled(D, 16, dtype=torch.float32).abs()
    b, c = filled(1, T, 1, 16), filled(1, T, 1, 16)
    g = fb.falcon_scan_bwd(x, dt, A, b, c, dy)
    far = lambda t: t[..., -n:].contiguous()  # noqa: E731
    g2 = fb.falcon_scan_bwd(far(x), far(dt), A[-n:].contiguous(), b, c, far(dy))
    assert torch.equal(g["dx"][..., -n:], g2["dx"]) and torch.equal(g["ddt"][..., -n:], g2["ddt"])
    assert torch.equal(g["dA"][-n:], g2["dA"])
