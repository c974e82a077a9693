"""The attention entry points' host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only).

The four attention sources are built host-only (no device code), as test_sanitizers.py builds the whole library, and
driven through the C ABI by tests/native/attn_abi_sanitize.c: refusals, workspace queries, and the planning of valid
calls over sizes up to the documented limits.
"""
import os

import pytest

from test_sanitizers import CSRC, ENV, NATIVE, ROOT, _run, _tool


def test_attention_host_side_under_asan_ubsan(tmp_path):
    hipcc = _tool(os.environ.get("HIPCC", "hipcc"), "/opt/rocm/bin/hipcc")
    clang = _tool("/opt/rocm/llvm/bin/clang", "clang")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined"]
    objs, names = [], set()
    for src in ("attn_api", "attn_prefill", "attn_backward", "attn_decode"):
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
    lib = str(tmp_path / "libattn_san.so")
    rc, out = _run([hipcc, "--offload-host-only", "-shared", "-fPIC"] + san + ["-o", lib] + objs + [str(tmp_path / "fatbin_stub.o")])
    assert rc == 0, out
    exe = str(tmp_path / "attn_abi_sanitize")
    rc, out = _run([clang, "-std=c99", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=undefined", "-I" + os.path.join(ROOT, "include"), "-o", exe,
                    os.path.join(NATIVE, "attn_abi_sanitize.c"), lib, "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-Wl,-rpath," + str(tmp_path)])
    assert rc == 0, out
    rc, out = _run([exe], env=ENV, timeout=200)
    if rc == 77:
        pytest.skip("a GPU is visible; the valid-call checks run only without one")
    assert rc == 0 and "all checks passed" in out, out
