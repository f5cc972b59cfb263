"""CPU test: the package may be imported before torch.  Both bring a HIP runtime into the process
unless the one that torch ships is there first, and with two the library finds no device."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("first,second", [("rope_partial_inplace_amd", "torch"),
                                          ("torch", "rope_partial_inplace_amd")])
def test_one_hip_runtime_whatever_is_imported_first(first, second):
    code = (f"import {first}; import {second}\n"
            "print(*{l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l})")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert len(r.stdout.split()) == 1, r.stdout
