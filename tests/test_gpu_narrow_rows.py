"""The way back for many narrow rows off the 16-byte boundaries: rows that share a
CTA."""

import numpy as np
import pytest
import torch

from tests import block_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("out_dtype", [0, 1, 2])
@pytest.mark.parametrize("M,K", [(2049, 1), (2049, 15), (2050, 129), (2051, 255), (2500, 257), (3001, 333), (2049, 340),
                                 (2053, 514), (2049, 1023)])
def test_many_narrow_rows_come_back(fmt, out_dtype, M, K):
    import quantized_fp8_attention_b200 as f
    q = R.random_microscaled(M, K, fmt, M + K, wide=True)
    held = torch.full((M * K + 64,), -77.0, dtype=f._OUT_DTYPE[out_dtype], device="cuda")
    got = f.mx_dequantize(q, out_dtype, out=held[: M * K].view(M, K))
    assert (held[M * K:] == -77.0).all()
    want = R.values(*R.held(q), fmt, K)
    # code * scale is exact in binary32; the row scale's product rounds once there
    # and the output once more
    half = torch.finfo(got.dtype).eps / 2 + (2.0 ** -24 if fmt == "nvfp4" else 0.0)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= half * 1.001 * np.abs(want) + (2.0 ** -25 if out_dtype == 2 else 0.0)).all()
