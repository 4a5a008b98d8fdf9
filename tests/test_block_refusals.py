"""Refusals of the microscaled and rotary functions that must not depend on the
calls before them, on the CPU."""

import pytest
import torch

import quantized_fp8_attention_b200 as fqa


def test_a_float_is_refused_whatever_was_asked_before_and_spoils_nothing_after():
    for first, then in ((4096.0, 4096), (8192, 8192.0)):
        for K in (first, then, first):
            if isinstance(K, float):
                with pytest.raises(ValueError, match="whole"):
                    fqa._mx_shapes(7, K, 0)
                with pytest.raises(ValueError, match="whole"):
                    fqa.alloc_microscaled(7, K, "mxfp8", "cpu")
            else:
                q = fqa.alloc_microscaled(7, K, "mxfp8", "cpu")
                assert q.codes.shape == (7, K) and all(type(n) is int for n in fqa._mx_shapes(7, K, 0)[0])
    for first, then in (((24, 104), (24.0, 104.0)), ((40.0, 88), (40, 88))):
        for axes in (first, then, first):
            if any(isinstance(a, float) for a in axes):
                with pytest.raises(ValueError, match="whole"):
                    fqa._axes_array(axes, False)
            else:
                assert list(fqa._axes_array(axes, False)) == list(axes)


def test_whole_numbers_of_other_types_serve():
    np = pytest.importorskip("numpy")
    q = fqa.alloc_microscaled(np.int64(130), np.int32(100), "nvfp4", "cpu")
    assert q.codes.shape == (130, 64) and q.scales.shape == (2, 2, 32, 4, 4) and type(q.cols) is int and q.cols == 100
