"""Seeded inputs and comparisons for the tests of the operators around the
recurrence.  Expected values come from oracle/block_oracle.py."""

import numpy as np
import torch

from delta_rule_recurrence_amd.inputs import as_f64

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
UNIT = 2.0 ** -24   # float32: half a step


def tolerance(dtype, depth):
    """Relative L2 bound of one result.

    Every float32 operation is off by at most UNIT of its value (the hardware's
    exp2, log2 and reciprocal by two).  A result is made by at most about 16
    operations and a chain of `depth` additions or products (the tokens a state
    has seen, the terms of a sum), whose errors add at most linearly; the
    inputs have random signs, so partial sums exceed the result by a small
    factor only, for which 4 stands.  A bfloat16 result adds its rounding,
    2^-8 of the value.
    """
    return 4 * (16 + depth) * UNIT + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)


def close(got, want, depth, what):
    """Finite where the oracle is, and within the tolerance as a whole."""
    g = as_f64(got)
    assert g.shape == want.shape, f"{what}: {g.shape} for {want.shape}"
    assert np.array_equal(np.isfinite(g), np.isfinite(want)), f"{what}: not finite"
    norm = np.linalg.norm(want)
    err = np.linalg.norm(g - want) / (norm if norm > 0 else 1.0)
    tol = tolerance(got.dtype, depth)
    print(f"{what}: {err:.2e} (at most {tol:.2e})", flush=True)
    assert err <= tol, f"{what}: relative error {err:.3e}, at most {tol:.3e}"


def draws(seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32, mean=0.0):
        return (mean + scale * torch.randn(*shape, generator=g)).to(dtype)

    return normal


def columns(t, pad=16):
    """The same values as columns of a wider projection whose other columns are
    NaN (a multiple of 8 elements aside, so the base stays 16-byte aligned)."""
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + 2 * pad,), float("nan"), dtype=t.dtype)
    wide[..., pad:pad + t.shape[-1]] = t
    return wide.cuda()[..., pad:pad + t.shape[-1]]


def f64(t):
    return None if t is None else as_f64(t)


def cuda(t):
    return None if t is None else t.cuda()


def pick(d, *names):
    return {n: d[n] for n in names}
