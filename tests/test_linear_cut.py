"""How packed calls of Linear Relation are cut (csrc/linear_cut.h) on the host: a small program compiled from the same
header walks offsets that ascend, descend and repeat, and checks that no segment leaves the list that the call has
room for and that no row is in two segments."""
import os
import subprocess

import pytest

from relation_token_mixing_gb300 import build as rbuild

HERE = os.path.dirname(os.path.abspath(__file__))
OUT = os.path.join(HERE, "_build", "linear_cut_check")


@pytest.fixture(scope="module")
def program():
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    cmd = [rbuild._nvcc(), *rbuild.ARCH, "-std=c++17", "-O2", "-I", rbuild.CSRC,
           os.path.join(HERE, "linear_cut_check.cu"), "-o", OUT]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return OUT


def test_no_offsets_lead_past_the_list(program):
    r = subprocess.run([program], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_requests_that_share_rows_would(program):
    """The walk notices: with every request's own offsets alone checked, repeated rows pass the list's end."""
    r = subprocess.run([program, "blind"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 1 and "segments" in r.stdout, r.stdout


def test_the_kernels_take_their_bounds_from_the_same_header():
    text = open(os.path.join(rbuild.CSRC, "linear_pool.cu")).read()
    assert "segments_of(sp, before, plan.seg_tokens)" in text and "span_between(" in text
    assert text.count("at + segs > plan.most_items") == 1  # the join's own
