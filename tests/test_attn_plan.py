"""How the attention backward deals out its work, checked on the host (CPU only).

tests/native/attn_plan_check.hip takes the plan's own header
(csrc/attn_backward_plan.h, the code that the kernels run) and compares it with
the definition in 64 bits, over random sizes and sizes at the documented limits.
It is built without device code, with UndefinedBehaviorSanitizer.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_08_amd", "csrc")


def test_backward_plan(tmp_path):
    hipcc = os.environ.get("HIPCC") or shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    exe = str(tmp_path / "attn_plan_check")
    r = subprocess.run([hipcc, "--offload-host-only", "-O1", "-g", "-std=c++17", "-Xarch_host", "-fsanitize=undefined",
                        "-Xarch_host", "-fno-sanitize-recover=undefined", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                        os.path.join(ROOT, "tests", "native", "attn_plan_check.hip"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout + r.stderr
