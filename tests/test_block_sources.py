"""What the sources of the overlapped kernels promise, read on the CPU."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_fp8_attention_b200", "csrc")


@pytest.mark.parametrize("name", ["rotary.cuh", "microscale.cuh", "matmul_mx.cuh"])
def test_overlapped_kernels_load_nothing_through_the_read_only_path(name):
    """They start while the kernel before them still writes what they read."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__ldg|\.nc\b|__restrict__|ldglobal", code)
