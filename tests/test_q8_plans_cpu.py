"""CPU tests of the 8-bit cache's and the page calls' launch plans (no GPU): tests/q8_plan_check.cpp,
compiled with the library's own plan sources, plain and under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only, g++)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rope_partial_inplace_amd", "csrc")
SAN = ["-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
       "-fno-sanitize-recover=all"]


@pytest.mark.parametrize("flags,rounds", [(["-O2"], "8000"), (SAN, "1000")], ids=["plain", "sanitized"])
def test_plans(tmp_path, flags, rounds):
    exe = str(tmp_path / "q8_plan_check")
    subprocess.run(["g++", "-std=c++17", *flags, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", "q8_plan_check.cpp"),
                    os.path.join(CSRC, "rope_q8_plan.cpp"), os.path.join(CSRC, "rope_pages_plan.cpp"),
                    "-o", exe], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe, rounds], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout[-2000:] + r.stderr[-4000:]
