"""Convolutions of more threads than one grid holds, on the CPU: the call comes
back with a status, in a child process with no visible device.  Its addresses
are fake and never dereferenced, so it never runs where a GPU is present."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALL = """
import ctypes, sys
sys.path.insert(0, {root!r})
from delta_rule_recurrence_amd import falcon as fb
lib = fb.load_library()
B, T, C, bf16, first = {case}
at = lambda i: ctypes.c_void_p((1 << 44) + i * (1 << 42))
p = fb.FalconConvProblem(B, T, C, 4, bf16, 1, C)
state = None if first else at(3)
print("status", lib.falcon_conv_fwd(ctypes.byref(p), at(0), at(1), at(2), state, at(4), at(5), at(6), None))
"""

# (B, T, C, bf16, without a state): every sequence's vectors together pass 2^32
CASES = [(65536, 1, 65537, 0, True), (262144, 1, 65537, 0, False), (1048576, 1, 32775, 0, True), (1 << 22, 1, 1 << 15, 1, False),
         (1 << 20, 1, 1 << 16, 0, True), (1 << 16, 5, 99999, 1, True), (1 << 16, 40, 65537, 0, True)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_a_convolution_of_more_threads_than_a_grid(case):
    if os.path.exists("/dev/kfd"):
        pytest.skip("a GPU is present: fake addresses must not reach it")
    env = dict(os.environ, HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="", CUDA_VISIBLE_DEVICES="")
    res = subprocess.run([sys.executable, "-c", CALL.format(root=ROOT, case=case)], env=env, capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, f"the process ended with {res.returncode}: {res.stderr[-500:]}"
    # valid arguments: the launch itself fails without a device
    assert res.stdout.split()[-1] in ("0", "-8"), res.stdout
