"""Norms of rows at the ends of binary32, as include/fqa.h states them."""

import numpy as np
import pytest
import torch

from tests import block_ref as R
from tests.test_gpu_microscale import check_norm, fqa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("K", [64, 4096, 4097, 20000])
def test_sums_of_squares_up_to_and_beyond_the_largest_number(fmt, K):
    f = fqa()
    g = torch.Generator(device="cuda").manual_seed(K)
    sign = torch.randint(0, 2, (4, K), device="cuda", generator=g) * 2.0 - 1.0
    x = sign * (1.0 + torch.rand(4, K, device="cuda", generator=g))
    # values of 1 to 2 times this: squares that add up to at most 2^126, or to more
    # than 2^129
    root = 2.0 ** np.floor(np.log2(2.0 ** 62 / np.sqrt(K)))
    x[:2] *= root
    x[2:] *= root * 16
    w = torch.ones(K, device="cuda")
    q, h = f.mx_rms_norm(x[:2], w, fmt, eps=1e-6)
    check_norm(x[:2], w, None, fmt, 1e-6, q, h, 2.0 ** -17)
    v = f.mx_dequantize(f.mx_rms_norm(x, w, fmt, eps=1e-6)[0], 1)
    assert (v[2:] == 0).all() and torch.equal(v[:2], f.mx_dequantize(q, 1))


def test_rotary_norm_of_such_heads_and_of_infinities():
    f = fqa()
    x = torch.randn(1, 4, 1, 128, device="cuda")
    clean = x.clone()
    x[0, 1] *= 2.0 ** 70
    x[0, 2, 0, 6], x[0, 3, 0, 9] = float("inf"), float("nan")
    rot = f.Rotary(torch.full((1, 1), 3, dtype=torch.int32, device="cuda"), (128,), q_weight=torch.ones(128, device="cuda"))
    y, want = f.rotary(x, None, rot)[0][0, :, 0], f.rotary(clean, None, rot)[0][0, :, 0]
    assert torch.equal(y[0], want[0]) and (y[1] == 0).all() and torch.isnan(y[3]).all()
    assert torch.isnan(y[2, 6:8]).all() and (y[2, :6] == 0).all() and (y[2, 8:] == 0).all()
    plain, plain_want = (f.rotary(t, None, rot._replace(q_weight=None))[0][0, :, 0] for t in (x, clean))
    assert not torch.isfinite(plain[2, 6:8]).any() and torch.equal(plain[2, 8:], plain_want[2, 8:])
    assert torch.isnan(plain[3, 8:10]).all() and torch.equal(plain[3, :8], plain_want[3, :8])
