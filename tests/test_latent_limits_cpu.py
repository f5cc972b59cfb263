"""CPU tests of the latent attention calls' limits (no kernel runs here)."""
import pytest

import rope_partial_inplace_amd as ra
from test_paged_latent_cpu import CALLS, HAS_GPU, INVALID, RUNTIME


@pytest.mark.parametrize("call", ["paged", "forward", "backward"])
def test_scales_whose_product_with_log2_e_leaves_float32_are_refused(call):
    for scale in (1e39, -1e300, 2.0 ** 128 / 1.4426, -2.0 ** 128 / 1.4426):
        assert CALLS[call]().run(scale=scale) == INVALID
        assert "scale" in ra.last_error()
    if not HAS_GPU:  # there a valid call would launch on host buffers
        for scale in (2.0 ** 126, -2.0 ** 127 * 0.99, 1e-300, -1e-45):
            assert CALLS[call]().run(scale=scale) == RUNTIME
