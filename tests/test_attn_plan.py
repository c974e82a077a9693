"""How the attention backward deals out its work, checked on the host (CPU only).

tests/native/attn_plan_check.hip takes the plan's own header
(csrc/attn_backward_plan.h, the code that the kernels run) and compares it with
the definition in 64 bits, over random sizes and sizes at the documented limits.
It is built without device code, with UndefinedBehaviorSanitizer.
"""
import os
import shutil
import subprocess
import time

import pytest

import gated_delta_rule_08_amd as gdr

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


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdr.library_path()):
        from gated_delta_rule_08_amd import build
        build.build()
    return gdr.load_library()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (32, 1), (32, 2), (32, 8)])
def test_backward_workspace_is_bounded(lib, dtype, Hq, Hkv):
    """Partial gradients take at most 256 MiB beside the 8 bytes of statistics for each query and head (and 2 KiB), on both sides of
    512 key blocks (65408 keys of one head), without and with a window."""
    for T in (300, 4096, 16384, 32768, 65408, 65409, 65500, 131072):
        for window in (0, 64, 4096):
            need = lib.gdr_attn_backward_workspace_bytes(dtype, 1, T, T, Hq, Hkv, 128, window, 0)
            assert 8 * T * Hq <= need <= 8 * (T * Hq + 4 * Hkv) + 2048 + (256 << 20), (T, window, need)


def test_planning_does_not_grow_with_the_length(lib):
    """The plan is formed on the host in every call: 469 key blocks take at most five times as long as 32 (twice
    here; block by block eleven times)."""
    def us(*shape):
        times = []
        for _ in range(40):
            t0 = time.perf_counter()
            for _ in range(25):
                lib.gdr_attn_backward_workspace_bytes(*shape)
            times.append(time.perf_counter() - t0)
        return min(times) / 25 * 1e6

    short, long = us(1, 1, 4096, 4096, 32, 8, 128, 0, 0), us(1, 1, 60000, 60000, 8, 1, 128, 256, 0)
    assert long <= 5 * short, (short, long)
