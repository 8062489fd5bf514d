"""The C ABI of the operators around the recurrence under the host sanitizers
(see test_host_sanitizers.py): tests/host_block_driver.py in a child process
with the ASan runtime preloaded and no visible device.  Never run where a GPU is
present: its fake addresses must not reach a device."""

import os
import subprocess
import sys

from delta_rule_recurrence_amd import build as B

from test_host_sanitizers import san_lib  # noqa: F401  (the fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_block_abi_under_host_sanitizers(san_lib):  # noqa: F811
    env = dict(os.environ)
    env.update(HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="", CUDA_VISIBLE_DEVICES="", LD_PRELOAD=B.asan_runtime(),
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "host_block_driver.py"), san_lib], env=env,
                         capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, f"driver failed ({res.returncode}):\n{res.stdout[-2000:]}\n{res.stderr[-6000:]}"
    assert "calls checked" in res.stdout
