"""Drives the C ABI of linear attention and of the residual update in the host-sanitised,
bounds-checked build (libfalcon_san.so) on a machine with no visible GPU: sizes,
workspaces, launch shapes and refusals of calls on fake device addresses, which are
never dereferenced.  Run by tests/test_host_sanitizers_linear_residual.py.  argv: path
of libfalcon_san.so.
"""

import ctypes
import itertools
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
from delta_rule_recurrence_amd import falcon as fb  # noqa: E402

lib = fb.load_library(sys.argv[1])
OK, HIP, WORKSPACE = 0, -8, -6
LAUNCHED = (OK, HIP)            # valid arguments: the launch itself fails without a device
NONE = ctypes.c_size_t(-1).value
calls = 0
at = 1 << 44


def fake(nbytes, there=True):
    """Distinct fake device addresses, each range followed by a gap."""
    global at
    if not there:
        return None
    a = at
    at += (max(int(nbytes), 1) + 4095) // 4096 * 4096 + (1 << 20)
    return a


def run(fn, p, *args, want=LAUNCHED):
    global calls
    calls += 1
    status = fn(ctypes.byref(p), *args, None)
    assert status in want, (fn.__name__, {f: getattr(p, f) for f, _ in p._fields_}, status)


def linear():
    for B, H, T, (dk, dv), bf16, heads in itertools.product((0, 1, 5, 300), (1, 3, 12), (0, 1, 64, 65, 2048, 100001),
                                                            ((16, 16), (32, 128), (64, 64), (128, 64), (128, 128)), (0, 1), (0, 1)):
        es, n, ns = 2 if bf16 else 4, B * T * H, B * H * dk * dv
        p = fb.FalconLinearProblem(B, H, T, dk, dv, bf16, heads, heads, heads, 0.5, H * dk + 8, H * dk, H * dv + 16)
        q, k, v = fake(B * T * (H * dk + 8) * es), fake(n * dk * es), fake(B * T * (H * dv + 16) * es)
        g, S0, ends = fake(H * 4), fake(ns * 4, heads), fake(B * 4, bf16)
        need = lib.falcon_linear_workspace_bytes(ctypes.byref(p))
        assert need != NONE
        args = [q, k, v, g, S0, ends, fake(n * dv * es), fake(ns * 4, not heads), fake(need) if need else None, need]
        run(lib.falcon_linear_fwd, p, *args)
        if need and n:
            run(lib.falcon_linear_fwd, p, *args[:-1], need - 1, want=(WORKSPACE,))
        run(lib.falcon_linear_step, p, q, k, v, g, fake(ns * 4), fake(B, heads), fake(B * H * dv * es))
        need = lib.falcon_linear_bwd_workspace_bytes(ctypes.byref(p))
        assert need != NONE
        args = [q, k, v, g, S0, ends, fake(n * dv * es), fake(ns * 4, bf16), fake(n * dk * 4), fake(n * dk * 4), fake(n * dv * 4),
                fake(H * 4, heads), fake(ns * 4, heads), fake(need) if need else None, need]
        run(lib.falcon_linear_bwd, p, *args)
        if need and n:
            run(lib.falcon_linear_bwd, p, *args[:-1], need - 1, want=(WORKSPACE,))


def residual():
    for B, T, (G, d), bf16, act, (post, pre), eight in itertools.product(
            (0, 1, 7), (0, 1, 33, 5000), ((1, 1), (5, 9), (12, 64), (40, 32), (1, 1001), (1, 8192), (8192, 1), (3, 2048)), (0, 1), (0, 3),
            ((1, 1), (0, 1), (1, 0)), (0, 1)):
        es, C = 2 if bf16 else 4, G * d
        n, steps = B * T * C, B * T * ((C + 31) // 32)
        p = fb.FalconResidualProblem(B, T, G, d, bf16, 1 - bf16, act, post, pre, 1e-6, C + 8 * act, C)
        y, gate, h = fake(B * T * (C + 24) * es), fake(n * es, act), fake(n * 4, bf16)
        wp, a, wn, ends = fake(C * 4, post), fake(C * 4, act), fake(C * 4), fake(B * 4, act)
        saved = ctypes.byref(fb.FalconSavedPointers(fake(n), fake(steps), fake(n, act), fake(steps, act)))
        h_out = fake(n * 4)
        run(lib.falcon_residual_fwd, p, y, gate, h, wp, a, wn, ends, h_out, fake(n * es), saved if eight else None)
        need = lib.falcon_residual_bwd_workspace_bytes(ctypes.byref(p))
        assert need != NONE
        first = (None, None, saved) if eight else (y, gate, None)
        args = [*first, h_out, wp, a, wn, ends, fake(n * 4, bf16), 0, fake(n * es), bf16, fake(n * 4), fake(n * 4), fake(n * 4, post),
                fake(C * 4), fake(C * 4), fake(C * 4, pre), fake(need) if need else None, need]
        run(lib.falcon_residual_bwd, p, *args)
        if need:
            run(lib.falcon_residual_bwd, p, *args[:-1], need - 1, want=(WORKSPACE,))


if __name__ == "__main__":
    linear()
    residual()
    print(f"host linear and residual driver: {calls} calls checked", flush=True)
