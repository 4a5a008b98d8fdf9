"""Rows off the 16-byte boundaries whose padded length fills the shared memory
that a launch has by default."""

import os
import subprocess
import sys

import pytest
import torch

from tests import block_ref as R
from tests.test_gpu_microscale import DT, check_norm, fqa, rand, same_as_reference

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rows_at_the_default_limit():
    """Padded to 12288 values by both widths of a scale word (12161, 12225 on), in
    single values and pairs, and a shifted view of 12288."""
    f = fqa()
    for dt in ("bf16", "f16", "f32"):
        for K in (12161, 12162, 12225, 12226, 12286, 12287):
            x, r = rand(2, K, dt, K, 1.0), rand(2, K, dt, K + 1, 1.0)
            w = (1 + 0.3 * torch.randn(K, device="cuda")).to(DT[dt])
            for fmt in R.FORMATS:
                same_as_reference(f.mx_quantize(x, fmt), x.double().cpu().numpy())
                q, h = f.mx_rms_norm(x, w, fmt, residual=r, eps=1e-5)
                check_norm(x, w, r, fmt, 1e-5, q, h, 2.0 ** -17)
        x = rand(2, 12300, dt, 1)[:, 1:12289]
        for fmt in R.FORMATS:
            same_as_reference(f.mx_quantize(x, fmt), x.double().cpu().numpy())


def test_rows_at_the_default_limit_of_shared_memory():
    """In a process of its own: a longer row of the same kernel raises the limit
    for all that follow."""
    run = subprocess.run([sys.executable, "-c", "from tests import test_gpu_row_lengths as t; t.rows_at_the_default_limit()"],
                         cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert run.returncode == 0, run.stderr[-2000:]
