"""Scalars at the ends of their ranges (CPU only: refused before any launch, or stopped at the device query)."""

import numpy as np
import pytest
import torch

from tests.test_cache_abi import CUDA, INVALID, NO_GPU, UNSUPPORTED, _attend, _call_attend, _msg, lib  # noqa: F401

LARGEST = float(np.finfo(np.float32).max)


def test_a_scale_that_overflows_in_units_of_log2_is_refused(lib):
    for scale in (LARGEST, 3e38, 2.4e38):  # times log2(e) these are infinite, and a score of 0 would be NaN
        assert _call_attend(lib, _attend(), scale=scale) == INVALID
        assert "scale" in _msg(lib)


@pytest.mark.skipif(not NO_GPU, reason="a valid call would launch on host memory")
def test_scales_within_the_range_are_served(lib):
    for scale in (1e-45, 1e-30, 1.0, 2.3e38):
        assert _call_attend(lib, _attend(dtype=torch.float32), scale=scale) in (UNSUPPORTED, CUDA), _msg(lib)
