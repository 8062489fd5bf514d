"""The norm's parameter gradients over many tokens."""

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,d", [(256, 8), (2, 1024), (1, 2048), (1, 4096)])
def test_sums_of_one_sign_over_many_tokens(G, d):
    """Gradients that all have one sign and size, whose rounding errors do not
    cancel.  x is one everywhere, so xhat = 1 / sqrt(1 + eps), dbias = tokens dy and
    dweight = dbias xhat.

    A thread of 512 workgroups adds up to 2048 tokens, 64 at a time and then those
    up to 32 sums: 64 + 32 float32 additions, each off by at most 2^-24 of a partial
    sum, none larger than the whole.  What joins the threads is in double.  The
    partial sums' and the result's roundings are two, and xhat has at most 4: its mean
    square and reciprocal root.
    """
    tokens = 1 << 20
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GiB of device memory")
    x = torch.ones(1, tokens, G * d, dtype=torch.bfloat16, device="cuda")
    dy = torch.full((1, tokens, G * d), 0.1, device="cuda")
    one = torch.ones(G * d, device="cuda")
    g = fb.falcon_norm_bwd(x, G, dy, one, one, eps=1e-6)
    dbias = tokens * float(torch.tensor(0.1, dtype=torch.float32))
    bound = (64 + 32 + 2 + 4) * 2.0 ** -24
    for name, want in (("dbias", dbias), ("dweight", dbias / (1 + 1e-6) ** 0.5)):
        err = float((g[name].double() / want - 1).abs().max())
        print(f"{name}: {err:.2e} (at most {bound:.2e})", flush=True)
        assert err <= bound, name
    del x, dy, g
    torch.cuda.empty_cache()
