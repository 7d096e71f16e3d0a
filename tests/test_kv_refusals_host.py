"""What the calls on the key-value cache refuse before any device work, beyond test_kv_host.py: arguments
whose products or sums overflow on the way to the kernels."""

import numpy as np
import pytest

from nvfp4_block_scaled_06_gb300 import _binding as B
from test_kv_host import REFUSED, attend, clib  # noqa: F401


@pytest.mark.parametrize("scale", [2.3e38, 2.0 ** 100, 1e-38])
def test_scales_that_the_kernels_can_hold(clib, scale):  # noqa: F811
    assert attend(clib, scale=scale) not in REFUSED


@pytest.mark.parametrize("scale", [2.4e38, 3.0e38, float(np.finfo(np.float32).max)])
def test_scales_whose_base_2_form_overflows(clib, scale):  # noqa: F811
    """The kernels multiply by scale * log2(e): infinite, it would make NaN of every score of 0."""
    assert np.isinf(np.float32(scale) * np.float32(1.4426950408889634))
    assert attend(clib, scale=scale) == B.ERR_INVALID_ARG
