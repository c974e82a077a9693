"""The copies to LDS write M0 in inline assembly, which the compiler cannot be told (M0 is a reserved register: a
clobber entry is refused with a warning).  The compiled attention kernels therefore use M0 nowhere else."""
import concurrent.futures
import os
import re
import subprocess

import pytest

from gated_delta_rule_08_amd import build


def m0_uses(path):
    """Instructions that name M0: (inside inline assembly, outside)."""
    inside, counts = False, [0, []]
    with open(path) as f:
        for line in f:
            if ";;#ASMSTART" in line or ";#ASMSTART" in line:
                inside = True
            elif "#ASMEND" in line:
                inside = False
            elif re.search(r"\bm0\b", line.split(";")[0]):
                if inside:
                    counts[0] += 1
                else:
                    counts[1].append(line.strip())
    return counts


def test_no_other_instruction_uses_m0(tmp_path):
    try:
        hipcc = build._hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")

    def compile_(name):
        out = str(tmp_path / (name + ".s"))
        r = subprocess.run([hipcc] + build.HIPFLAGS + ["-S", "--offload-device-only", os.path.join(build.CSRC, name + ".hip"), "-o", out],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return m0_uses(out)

    with concurrent.futures.ThreadPoolExecutor(3) as pool:
        for inside, outside in pool.map(compile_, ("attn_prefill", "attn_backward", "attn_decode")):
            assert inside > 0 and not outside, outside[:5]
