"""Drives the C ABI of the operators around the recurrence in the host-sanitised,
bounds-checked build (libfalcon_san.so) on a machine with no visible GPU: sizes,
workspaces, launch shapes and refusals of thousands of calls on fake device
addresses, which are never dereferenced.  Run by
tests/test_host_sanitizers_block.py.  argv: path of libfalcon_san.so.
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


class Fake:
    """Distinct fake device addresses, each range followed by a gap."""

    def __init__(self):
        self.next = 1 << 44

    def __call__(self, nbytes, there=True):
        if not there:
            return None
        a = self.next
        self.next += (max(int(nbytes), 1) + 4095) // 4096 * 4096 + (1 << 20)
        return a


def run(fn, p, *args, want=LAUNCHED):
    global calls
    calls += 1
    status = fn(ctypes.byref(p), *args, None)
    assert status in want, (fn.__name__, {f: getattr(p, f) for f, _ in p._fields_}, status)


def short(fn, p, args, need):
    """The same call with a workspace one byte short."""
    if need > 0:
        run(fn, p, *args[:-1], need - 1, want=(WORKSPACE,))


def conv(fake):
    for B, T, C, W, bf16, extra in itertools.product((0, 1, 3, 64), (0, 1, 7, 2048, 100001), (1, 7, 64, 1001, 4608), (2, 3, 4),
                                                     (0, 1), (0, 8)):
        es, n, ns = 2 if bf16 else 4, B * T * C, B * (W - 1) * C
        p = fb.FalconConvProblem(B, T, C, W, bf16, 1, C + extra)
        x, w, b, s = fake(B * T * (C + extra) * es), fake(C * W * 4), fake(C * 4), fake(ns * es, bf16)
        ends = fake(B * 4, extra)
        run(lib.falcon_conv_fwd, p, x, w, b, s, ends, fake(n * es), fake(ns * es, extra))
        run(lib.falcon_conv_step, p, fake(B * (C + extra) * es), w, b, fake(ns * es), fake(B, extra), fake(B * C * es))
        need = lib.falcon_conv_bwd_workspace_bytes(ctypes.byref(p))
        assert need != NONE
        args = [x, w, b, s, ends, fake(n * 4), 0, fake(ns * 4, extra), fake(n * 4), fake(C * W * 4), fake(C * 4, bf16), fake(ns * 4),
                fake(need), need]
        run(lib.falcon_conv_bwd, p, *args)
        short(lib.falcon_conv_bwd, p, args, need)


def norm(fake):
    for B, T, (G, d), bf16, (xh, yh), act in itertools.product((0, 1, 5), (0, 1, 33, 4096), ((1, 1), (5, 9), (12, 64), (40, 32), (3, 1001),
                                                                                            (1, 4096), (32, 128)),
                                                               (0, 1), ((0, 0), (0, 1), (1, 0), (1, 1)), (0, 2)):
        es, C = 2 if bf16 else 4, G * d
        n = B * T * C
        p = fb.FalconNormProblem(B, T, G, d, bf16, act, 1, xh, yh, 1e-6, 1.0, C + 8 * (1 - xh))
        x, w, b = fake(B * T * (C + 8) * es), fake(C * 4, act), fake(C * 4)
        run(lib.falcon_norm_fwd, p, x, w, b, fake(n * es))
        need = lib.falcon_norm_bwd_workspace_bytes(ctypes.byref(p))
        assert need != NONE
        args = [x, w, b, fake(n * 4), 0, fake(n * 4), fake(C * 4, act), fake(C * 4), fake(need), need]
        run(lib.falcon_norm_bwd, p, *args)
        short(lib.falcon_norm_bwd, p, args, need)


def scan(fake):
    for B, T, (D, G), N, bf16, extra in itertools.product((0, 1, 8), (0, 1, 65, 2048, 100001), ((1, 1), (96, 1), (250, 2), (768, 4)),
                                                          (8, 16, 32, 64), (0, 1), (0, 8)):
        es, n, ns = 2 if bf16 else 4, B * T * D, B * D * N
        wide, shared = D + extra, G * N + extra
        p = fb.FalconScanProblem(B, T, D, N, G, bf16, 1, wide, wide, wide, shared, shared)
        x, dt, A, Bm, Cm = fake(B * T * wide * es), fake(B * T * wide * es), fake(D * N * 4), fake(B * T * shared * es), fake(B * T * shared * es)
        skip, bias, z, S0, ends = fake(D * 4, extra), fake(D * 4), fake(B * T * wide * es, bf16), fake(ns * 4, extra), fake(B * 4, bf16)
        first = (x, dt, A, Bm, Cm, skip, bias, z)
        need = lib.falcon_scan_workspace_bytes(ctypes.byref(p))
        assert need != NONE
        args = [*first, S0, ends, fake(n * es), fake(ns * 4), fake(need) if need else None, need]
        run(lib.falcon_scan_fwd, p, *args)
        if n:
            short(lib.falcon_scan_fwd, p, args, need)
        run(lib.falcon_scan_step, p, *first, fake(ns * 4), fake(B, extra), fake(B * D * es))
        need = lib.falcon_scan_bwd_workspace_bytes(ctypes.byref(p))
        assert need != NONE
        args = [*first, S0, ends, fake(n * 4), 0, fake(ns * 4, extra), fake(n * 4), fake(n * 4), fake(n * 4), fake(D * N * 4),
                fake(B * T * G * N * 4), fake(B * T * G * N * 4), fake(D * 4), fake(D * 4, extra), fake(ns * 4), fake(need), need]
        run(lib.falcon_scan_bwd, p, *args)
        short(lib.falcon_scan_bwd, p, args, need)


if __name__ == "__main__":
    fake = Fake()
    conv(fake)
    norm(fake)
    scan(fake)
    print(f"host block driver: {calls} calls checked", flush=True)
