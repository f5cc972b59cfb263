"""CPU tests of single cases of the 8-bit cache's and the page calls' launch plans (no GPU):
tests/q8_edge_check.cpp, compiled with the library's own plan sources under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only, g++)."""
import os
import subprocess

import pytest
import torch

import rope_partial_inplace_amd as ra
from test_q8_plans_cpu import CSRC, ROOT, SAN


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("q8") / "q8_edge_check")
    subprocess.run(["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", "q8_edge_check.cpp"),
                    os.path.join(CSRC, "rope_q8_plan.cpp"), os.path.join(CSRC, "rope_pages_plan.cpp"),
                    "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("check", ["append_no_values", "append_long_blocks", "fork_layouts", "interleaved_caches"])
def test_plan(program, check):
    r = subprocess.run([program, check], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout[-2000:] + r.stderr[-4000:]


def test_caches_as_pages():
    """Whole pages: the same memory with one dimension a page, whatever the order of the others."""
    x = torch.arange(5 * 2 * 3 * 4, dtype=torch.int64).view(5, 2, 3, 4)
    for t in (x, x.permute(0, 3, 1, 2), x[::2], x[1:].transpose(1, 2), x[:, 1], x[:1], x[:, :, :, :1][:, :1, :1]):
        y = ra._as_pages(t)
        assert y.dim() == 2 and y.data_ptr() == t.data_ptr() and y.shape[0] == t.shape[0]
        for a, b in zip(t, y):
            assert sorted(a.flatten().tolist()) == b.tolist() and y.stride(1) == 1
    for t in (x[:, :, :2], x[..., 1:], x[..., ::2], x[:, :1].expand(5, 2, 3, 4)):
        with pytest.raises(ra.RopeError) as e:
            ra._as_pages(t)
        assert e.value.code == ra.ROPE_ERR_PARAM_INVALID
    one, none = torch.zeros(7), torch.zeros(3, 0, 4)
    assert ra._as_pages(one) is one and ra._as_pages(none) is none
    with pytest.raises(ra.RopeError):  # host memory
        ra.PageCaches([], whole=[x])
