"""The stream written over itself with another type or row stride is refused (CPU: no call here reaches a launch)."""
import ctypes

import pytest

import post_weight_quantization_accum_amd as P
from post_weight_quantization_accum_amd import _lib

FAKE = 0x1000          # never dereferenced


@pytest.mark.parametrize("x_dtype,h_dtype,ld_x,ld_h", [(0, 2, 64, 64), (2, 0, 64, 64), (1, 2, 64, 64), (2, 2, 64, 80), (0, 0, 80, 64)])
def test_another_layout_in_place(x_dtype, h_dtype, ld_x, ld_h):
    norm = _lib.Norm(_lib.NORM_RMS, 1e-6, 1.0, _lib.F32, None, None, None, None, 0)
    call = lambda h: P.load().gptq_residual_norm(ctypes.byref(norm), 4, 64, FAKE, x_dtype, ld_x, None, 0, 64, h, h_dtype, ld_h, None, 0,
                                                 64, None)
    assert call(FAKE) == _lib.ERR_INVALID_ARG
    assert call(None) == _lib.OK                         # nothing to write
