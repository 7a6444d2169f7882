"""Sizes past what one launch can hold are refused in words, before any launch."""

import ctypes

from expert_ffn_layer_top_amd import _lib

UNSUPPORTED = 2


def test_sizes_past_one_launch():
    L = _lib.lib
    p = ctypes.c_void_p(0x1000)
    assert L.moe_fp8b_quantize_rows(p, None, 1 << 25, 1024, 1, p, p, None) == UNSUPPORTED     # 2^32 threads
    assert b"2^32" in L.moe_last_error_string()
    T = (1 << 28) - 63
    assert L.moe_route_scored(p, None, T, 4, 1, 0, 1, 1, 1, 1, 1.0, p, p, None, p, p, None, 0, p, None, p, 1 << 62,
                              None) == UNSUPPORTED
    assert b"2^28" in L.moe_last_error_string()
    assert L.moe_route_scored_bwd(p, p, p, T, 4, 1, 0, 1, 1.0, p, None) == UNSUPPORTED
