"""nvfp4 products whose row scales lie at the ends of binary32 and whose results
do not."""

import numpy as np
import pytest
import torch

from tests import block_ref as R
from tests.test_gpu_mx_matmul import bound, fqa, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 260, 320), (5, 130, 4096), (40, 200, 96), (100, 257, 1056), (1500, 2048, 288),
                                   (1333, 2111, 2080)])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("whole", [False, True])
def test_results_in_range_of_row_scales_at_the_ends(M, N, K, bias, whole):
    f = fqa()
    a, b = R.random_microscaled(M, K, "nvfp4", 1, wide=True), R.random_microscaled(N, K, "nvfp4", 2, wide=True)
    g = np.random.default_rng(M)
    # row scales from 2^-149 to 2^127; `whole`: powers of two, as quantization
    # chooses them, else with odd fractions; plain rows among them
    def scales(n):
        e = g.choice([-149, -140, -126, -120, -100, -81, -80, -79, -20, 0, 20, 79, 80, 81, 100, 120, 126], n)
        s = 2.0 ** e * (1.0 if whole else g.uniform(1.0, 2.0, n))
        return torch.from_numpy(s.astype(np.float32)).cuda()
    near = a._replace(row_scale=torch.ones(M, device="cuda")), b
    a, b = a._replace(row_scale=scales(M)), b._replace(row_scale=scales(N))
    bv = torch.randn(N, device="cuda") if bias else None
    y, mag = reference(a, b, bv)
    out = f.mx_matmul(a, b, bias=bv, out_dtype=1).double()
    # of magnitudes that a sum of K products cannot carry past the largest number;
    # below the smallest normal one the steps are 2^-149
    sure = mag < 2.0 ** 126
    err = (out - y).abs()
    lim = bound(y, mag, K, torch.float32) + 2.0 ** -149
    assert sure.double().mean() > 0.5
    assert (err[sure] <= lim[sure]).all(), float((err / lim)[sure].max())
    # infinite where even a result that is off by its bound (products of both signs
    # may cancel to far less than their magnitude) would lie beyond the largest number
    beyond = y.abs() - lim > 2.0 ** 128
    assert torch.isinf(out[beyond]).all() and not torch.isnan(out).any()
    # a row's results do not depend on its neighbours' scales
    mixed = near[0]._replace(row_scale=torch.where(torch.arange(M, device="cuda") % 2 == 0, 1.0, a.row_scale))
    plain = f.mx_matmul(near[0], near[1], bias=bv, out_dtype=1)
    assert torch.equal(f.mx_matmul(mixed, near[1], bias=bv, out_dtype=1)[::2], plain[::2])
