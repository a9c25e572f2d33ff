"""Edges of libbeamattn.so and its binding that need no GPU: every call below is
refused on the host."""
import ctypes

import pytest

import beam_search_step_amd as bs
from beam_search_step_amd import attn


@pytest.mark.parametrize("scale", [1e-50, 1e-38, 1e30])
def test_scales_that_fp32_does_not_hold_are_refused(scale):
    """Below 1e-37 scale * log2(e) loses bits or is zero, and zero times the -inf of a
    key that is not seen is NaN."""
    h = ctypes.c_void_p(123)
    L = bs.attn_library()
    for create, cfg in ((L.bs_cache_attn_create, attn.bs_cache_attn_config(1, 1, 1, 1, 1, 64, 16, 1, 0, 1, scale)),
                        (L.bs_cross_attn_create, attn.bs_cross_attn_config(1, 1, 1, 1, 64, 8, 1, scale))):
        assert create(ctypes.addressof(cfg), None, ctypes.addressof(h)) == bs.BS_EINVAL
        assert h.value is None
