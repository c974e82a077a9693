"""The host code of the operators around the attention layers under AddressSanitizer and UndefinedBehaviorSanitizer, and
their kernels' use of M0 (CPU only).

The sources are built host-only, as test_attn_sanitizers.py does, and driven through the C ABI by
tests/native/serving_abi_sanitize.c.
"""
import os
import subprocess

import pytest

from gated_delta_rule_08_amd import build
from test_attn_m0 import m0_uses
from test_sanitizers import CSRC, ENV, NATIVE, ROOT, _run, _tool


def test_host_side_under_asan_ubsan(tmp_path):
    hipcc = _tool(os.environ.get("HIPCC", "hipcc"), "/opt/rocm/bin/hipcc")
    clang = _tool("/opt/rocm/llvm/bin/clang", "clang")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined"]
    objs, names = [], set()
    for src in ("attn_serving_api", "attn_rope", "attn_pages", "attn_mx4"):
        obj = str(tmp_path / (src + ".o"))
        rc, out = _run([hipcc, "--offload-host-only", "-O1", "-g", "-fPIC", "-std=c++17", "-fno-omit-frame-pointer"] + san +
                       ["-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-c", os.path.join(CSRC, src + ".hip"), "-o", obj])
        assert rc == 0, out
        rc, out = _run(["nm", "-u", obj])
        assert rc == 0, out
        names |= {ln.split()[-1] for ln in out.splitlines() if "__hip_fatbin_" in ln}
        objs.append(obj)
    # an empty offload bundle stands in for each object's absent device code
    stub = tmp_path / "fatbin_stub.c"
    stub.write_text("".join('const char %s[32] __attribute__((aligned(4096))) = "__CLANG_OFFLOAD_BUNDLE__";\n' % n
                            for n in sorted(names)))
    rc, out = _run([clang, "-c", "-fPIC", str(stub), "-o", str(tmp_path / "fatbin_stub.o")])
    assert rc == 0, out
    lib = str(tmp_path / "libserving_san.so")
    rc, out = _run([hipcc, "--offload-host-only", "-shared", "-fPIC"] + san + ["-o", lib] + objs + [str(tmp_path / "fatbin_stub.o")])
    assert rc == 0, out
    exe = str(tmp_path / "serving_abi_sanitize")
    rc, out = _run([clang, "-std=c99", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=undefined", "-I" + os.path.join(ROOT, "include"), "-o", exe,
                    os.path.join(NATIVE, "serving_abi_sanitize.c"), lib, "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-Wl,-rpath," + str(tmp_path)])
    assert rc == 0, out
    rc, out = _run([exe], env=ENV, timeout=200)
    if rc == 77:
        pytest.skip("a GPU is visible; the valid-call checks run only without one")
    assert rc == 0 and "all checks passed" in out, out


def test_no_other_instruction_of_the_mx4_kernels_uses_m0(tmp_path):
    try:
        hipcc = build._hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    out = str(tmp_path / "attn_mx4.s")
    r = subprocess.run([hipcc] + build.HIPFLAGS + ["-S", "--offload-device-only", os.path.join(build.CSRC, "attn_mx4.hip"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    inside, outside = m0_uses(out)
    assert inside > 0 and not outside, outside[:5]
