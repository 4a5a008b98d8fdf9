"""The 64-bit reference of the microscaled formats and of the rotary positions
against hand-worked cases (CPU)."""

import numpy as np
import torch

from tests import block_ref as R


def test_tables():
    assert R.E4M3[-1] == 448 and len(R.E4M3) == 127 and R.E4M3[8] == 2.0 ** -6 and R.E4M3[1] == 2.0 ** -9
    e4m3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.E4M3, e4m3)


def test_nearest_takes_ties_to_the_even_code_and_saturates():
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 100.0, 0.2501])
    assert R.nearest(x, R.E2M1).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 1]


def test_mx_scale_is_the_smallest_power_that_does_not_saturate():
    for amax, fmt, e in ((448.0, "mxfp8", 0), (449.0, "mxfp8", 1), (224.0, "mxfp8", -1), (6.0, "mxfp4", 0),
                         (6.01, "mxfp4", 1), (3.0, "mxfp4", -1), (1e-45, "mxfp4", -127), (0.0, "mxfp8", -127)):
        x = np.zeros((1, 32))
        x[0, 5] = amax
        codes, b, row = R.quantize(x, fmt)
        assert b[0, 0] == e + 127 and row is None, (amax, fmt)
    codes, b, _ = R.quantize(np.array([[3.0, -6.0, 0.75] + [0.0] * 29]), "mxfp4")
    assert codes[0, :4].tolist() == [5, 15, 2, 0] and b[0, 0] == 127


def test_nvfp4_by_hand():
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1], x[0, 16] = 2688.0, 224.0, 3.0
    codes, b, row = R.quantize(x, "nvfp4")
    # row scale 1; the first block's scale 448 (0x7E): 2688 -> 6, 224 = 0.5 * 448; the second's 0.5 (0x30)
    assert row[0] == 1.0 and b[0].tolist() == [0x7E, 0x30]
    assert codes[0, :2].tolist() == [7, 1] and codes[0, 16] == 7
    assert np.array_equal(R.values(codes, b, row, "nvfp4"), x)


def test_non_finite_blocks_stand_for_nan():
    x = np.ones((2, 64))
    x[0, 40] = np.inf
    for fmt in R.FORMATS:
        v = R.values(*R.quantize(x, fmt), fmt)
        assert np.isnan(v[0, 32:]).all() and np.isfinite(v[1]).all()
        assert np.isnan(v[0, :32]).all() == (fmt == "nvfp4")


def test_rotary_by_hand():
    x = torch.zeros(1, 1, 1, 128)
    x[..., 0], x[..., 64] = 1.0, 2.0
    pos = torch.tensor([[3.0]])
    y = R.rotary(x, pos, (128,), split=True)
    assert np.allclose([y[0, 0, 0, 0], y[0, 0, 0, 64]], [np.cos(3) - 2 * np.sin(3), np.sin(3) + 2 * np.cos(3)])
    y = R.rotary(x, torch.tensor([[5.0, 7.0]]), (64, 64))
    assert np.allclose([y[0, 0, 0, 0], y[0, 0, 0, 1]], [np.cos(5), np.sin(5)])
    assert np.allclose([y[0, 0, 0, 64], y[0, 0, 0, 65]], [2 * np.cos(7), 2 * np.sin(7)])
    back = R.rotary(torch.from_numpy(y), torch.tensor([[5.0, 7.0]]), (64, 64), inverse=True)
    assert np.allclose(back, x.numpy())
