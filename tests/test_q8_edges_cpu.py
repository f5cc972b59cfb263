"""CPU tests of single cases of the 8-bit cache's and the page calls' launch plans (no GPU):
tests/q8_edge_check.cpp, compiled with the library's own plan sources under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only, g++)."""
import os
import subprocess

import pytest

from test_q8_plans_cpu import CSRC, ROOT, SAN


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("q8") / "q8_edge_check")
    subprocess.run(["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", "q8_edge_check.cpp"),
                    os.path.join(CSRC, "rope_q8_plan.cpp"), os.path.join(CSRC, "rope_pages_plan.cpp"),
                    "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("check", ["append_no_values", "append_long_blocks"])
def test_plan(program, check):
    r = subprocess.run([program, check], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout[-2000:] + r.stderr[-4000:]
