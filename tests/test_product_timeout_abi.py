"""Refusals of the check of the products' waits, on the host."""

import ctypes

import pytest


@pytest.mark.parametrize("rank,stage", [(-2, 0), (8, 0), (0, -1), (0, (1 << 24) + 1)])
def test_refusals(rank, stage):
    from quantized_fp8_attention_b200 import build
    import quantized_fp8_attention_b200 as fqa
    build.build()
    L = fqa.lib()
    P, I = ctypes.c_void_p, ctypes.c_int
    L.fqa_debug_mx_matmul_timeout.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P, I, I, I, P]
    ok = P(0x10000)
    assert L.fqa_debug_mx_matmul_timeout(ok, ok, ok, ok, ok, ok, None, 4, 8, 64, 2, ok, 0, rank, stage, None) == 1
    # and the product's own
    assert L.fqa_debug_mx_matmul_timeout(None, ok, ok, ok, ok, ok, None, 4, 8, 64, 2, ok, 0, 0, 0, None) == 1
    assert L.fqa_debug_mx_matmul_timeout(ok, ok, ok, ok, ok, ok, None, 0, 8, 64, 2, ok, 0, 0, 0, None) == 0
