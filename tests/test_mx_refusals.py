"""Further refusals of the cache and attention entry points (CPU: no call here reaches a launch)."""
import pytest
import torch

import post_weight_quantization_accum_amd as P
from post_weight_quantization_accum_amd import _lib
from test_mx_oracle import BAD, _attend, _c


def test_scales_outside_their_range():
    """8 / scale and scale * log2(e) are held in float32: neither may overflow."""
    for scale in (2.0 ** -101, 1e-38, 1e-45, 2.0 ** 101, 3e38, -1.0):
        assert _attend(_c(), sc=scale) == BAD, scale
    for scale in (2.0 ** -100, 2.0 ** 100):
        assert _attend(_c(), sc=scale, n=0) == _lib.OK and _attend(_c(), sc=scale, mp=4096) == _lib.ERR_WORKSPACE
