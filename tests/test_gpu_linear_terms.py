"""Linear attention in bfloat16: what is float32 inside (decayed scores, states, what is
written into them) keeps float32's bits, so an output is rounded once."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

from block_utils import UNIT, draws, f64

pytestmark = pytest.mark.gpu


def near_ties(*shape, seed):
    """Float32 numbers of 24 bits, half of them just above the middle of two neighbouring
    bfloat16 numbers and half just below: (odd) 2^14 + 1 or - 1, whose last bit decides the
    rounding, of either sign."""
    g = torch.Generator().manual_seed(seed)
    pick = lambda lo, hi: torch.randint(lo, hi, shape, generator=g)  # noqa: E731
    odd, off, sign = 2 * pick(128, 256) + 1, 2 * pick(0, 2) - 1, 2 * pick(0, 2) - 1
    return odd, off, sign


# one tile a head, and several of one and of several chunks
TILES = [(1, 40), (1, 700), (150, 700)]


@pytest.mark.parametrize("B,T", TILES)
@pytest.mark.parametrize("dk,dv", [(16, 32), (64, 64), (128, 128)])
def test_a_state_is_read_with_all_its_bits(dk, dv, B, T):
    """Queries that pick a row of a state that nothing is added to."""
    B = min(B, 50) if dk == 128 else B
    odd, off, sign = near_ties(B, 2, dk, dv, seed=1)
    S0 = (sign * (odd * 2 ** 14 + off)).float()
    pick = torch.arange(T) % dk
    q = torch.eye(dk)[pick].expand(B, 2, T, dk).contiguous().bfloat16().cuda()
    none = torch.zeros(2, device="cuda")
    z = lambda d: torch.zeros(B, 2, T, d, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o, S_T = fb.falcon_linear_fwd(q, z(dk), z(dv), none, S0=S0.cuda())
    assert torch.equal(S_T.cpu(), S0)
    assert torch.equal(o.cpu(), S0.bfloat16()[:, :, pick])


@pytest.mark.parametrize("B,T", TILES)
@pytest.mark.parametrize("dk,dv", [(16, 32), (64, 64), (128, 128)])
def test_scores_enter_with_all_their_bits(dk, dv, B, T):
    """Keys at the chunks' starts, each in one score with a query, and values of one."""
    B = min(B, 50) if dk == 128 else B
    odd, off, sign = near_ties(B, 2, T, seed=2)
    k = torch.zeros(B, 2, T, dk)
    first = torch.arange(T) % 64 == 0
    # (odd 2^14 = (odd - 1) 2^14 + 2^14, each of 8 bits)
    k[..., 0], k[..., 1], k[..., 2] = (odd - 1) * 2 ** 14, 2 ** 14, off
    k *= (sign * first)[..., None]
    q = torch.zeros(B, 2, T, dk)
    q[..., :3] = 1
    v = torch.ones(B, 2, T, dv)
    # one chunk without a decay: every query reads the one score
    score = (sign * (odd * 2 ** 14 + off)).float()
    o, _ = fb.falcon_linear_fwd(q[:, :, :64].contiguous().bfloat16().cuda(), k[:, :, :64].contiguous().bfloat16().cuda(),
                                v[:, :, :64].contiguous().bfloat16().cuda(), torch.zeros(2, device="cuda"))
    assert torch.equal(o.cpu(), score[:, :, :1, None].bfloat16().expand(o.shape))
    # a longer prompt that keeps nothing: the tokens that open a chunk read their own
    o, _ = fb.falcon_linear_fwd(q.bfloat16().cuda(), k.bfloat16().cuda(), v.bfloat16().cuda(),
                                torch.full((2,), -float("inf"), device="cuda"))
    assert torch.equal(o[:, :, first].cpu(), score[:, :, first, None].bfloat16().expand(B, 2, int(first.sum()), dv))


@pytest.mark.parametrize("B,H,T,tiles", [(1, 2, 192, 1), (50, 2, 1000, 6), (200, 2, 400, 1)])
def test_what_is_written_into_a_state_keeps_its_bits(B, H, T, tiles):
    """One token of a chunk writes, a token a chunk behind reads: the value times its decay.

    Every output is off by its own rounding, half a step, and by float32's before it: the
    decay is a product of at most five powers, each off by 2 UNIT, whose exponents (at most
    4.4 together, rounded twice, of a base rounded once) add 3 x 0.7 x 4.4 UNIT, and of at
    most six products: under 32 UNIT.  (Two bfloat16 terms keep 2^-17, 128 UNIT.)"""
    dk, dv = 16, 32
    n = draws(5)
    need = fb.falcon_linear_workspace_bytes(fb.FalconLinearProblem(B, H, T, dk, dv, 1, 1, 1, 1, 1.0, H * dk, H * dk, H * dv))
    assert need == (B * H * tiles * dk * dv * 4 if tiles > 1 else 0)
    decay = torch.tensor([-0.01, -0.0373])
    chunks, k, q, v = T // 64, torch.zeros(B, H, T, dk), torch.zeros(B, H, T, dk), n(B, H, T, dv, dtype=torch.bfloat16)
    wrote, reads = [], []
    for c in range(min(chunks - 1, dk)):         # a key of its own each
        w, r = 64 * c + (11 * c + 5) % 64, 64 * (c + 1) + 17
        k[:, :, w, c] = 1
        q[:, :, r, c] = 1
        wrote.append(w), reads.append(r)
    o, _ = fb.falcon_linear_fwd(q.bfloat16().cuda(), k.bfloat16().cuda(), v.cuda(), decay.cuda())
    gap = np.array(reads) - np.array(wrote)
    want = f64(v)[:, :, wrote] * np.exp(f64(decay)[:, None, None] * gap[:, None])
    got = f64(o)[:, :, reads]
    half = np.exp2(np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126))) - 8)
    over = np.abs(got - want) - half
    print(f"{T} {tiles}: {(over / np.abs(want).clip(1e-30)).max() / UNIT:.1f} UNIT over half a step", flush=True)
    assert np.all(over <= 32 * UNIT * np.abs(want))
