"""The paged forward's schedule (csrc/paged_schedule.cuh) on the host: a small program compiled from the same header
compares the closed form of the places before each row tile with direct summation, over groups, cached lengths,
new tokens and the kernels' tile sizes."""
import os
import subprocess

from relation_token_mixing_gb300 import build as rbuild

HERE = os.path.dirname(os.path.abspath(__file__))
OUT = os.path.join(HERE, "_build", "paged_schedule_check")


def test_places_equal_direct_summation():
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    src = os.path.join(HERE, "paged_schedule_check.cu")
    cmd = [rbuild._nvcc(), *rbuild.ARCH, "-std=c++17", "-O2", "-I", rbuild.CSRC, src, "-o", OUT]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([OUT], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
