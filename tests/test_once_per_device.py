"""Steps that each device needs once (csrc/once_per_device.h), on the host with a fake step, and that the paged kernels
raise their shared-memory limit through it and not once a process."""
import os
import re
import subprocess

import pytest

from relation_token_mixing_gb300 import build as rbuild

HERE = os.path.dirname(os.path.abspath(__file__))
OUT = os.path.join(HERE, "_build", "once_per_device_check")


def test_each_device_once_and_again_after_an_error():
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    cmd = [rbuild._nvcc(), *rbuild.ARCH, "-std=c++17", "-O2", "-I", rbuild.CSRC,
           os.path.join(HERE, "once_per_device_check.cu"), "-o", OUT]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([OUT], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


@pytest.mark.parametrize("name", ["paged_few.cu", "paged_tc.cu", "paged_f32.cu"])
def test_paged_kernels_keep_no_flag_for_the_whole_process(name):
    text = open(os.path.join(rbuild.CSRC, name)).read()
    assert "call_once" not in text and len(re.findall(r"\bcudaFuncSetAttribute\b", text)) == 0
    assert len(re.findall(r"\ballow_dynamic_smem\(", text)) == 1
