"""Waits of the products that run into their limit: the call reports it, waits for
its own copies and products in flight, and leaves everything usable."""

import time

import pytest
import torch

from tests import block_ref as R

pytestmark = pytest.mark.gpu


def fqa():
    import quantized_fp8_attention_b200 as f
    return f


# one CTA a tile, wider tiles, clusters of eight CTAs that share K, pairs of CTAs
# with one and with several tiles each
SIZES = [(100, 300, 2048), (40, 128, 1024), (1, 256, 8192), (1500, 2048, 2048), (3000, 4096, 1056)]


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_waits_that_run_out(M, N, K, fmt):
    f = fqa()
    a, b = R.random_microscaled(M, K, fmt, 1), R.random_microscaled(N, K, fmt, 2)
    want = f.mx_matmul(a, b, out_dtype=1)
    held = torch.full((M * N + 256,), -77.0, device="cuda")
    out = held[: M * N].view(M, N)
    torch.cuda.synchronize()
    assert f.fqa_debug_status()[0] == f.FQA_OK
    gave_up = 0
    for rank in (-1, 0, 1, 7):
        for stage in (0, 1, 2, 3, 4, 5, 6, 9, 13, 1 << 24):
            out.fill_(-77.0)
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            assert f.fqa_debug_mx_matmul_timeout(a, b, out, 1, rank, stage) == f.FQA_OK
            st = f.fqa_debug_status()[0]
            # a wait for something in flight that never came would take its own
            # limit of 1.5 s
            assert time.perf_counter() - t0 < 1.0, (rank, stage)
            assert st in (f.FQA_OK, f.FQA_ERR_TIMEOUT)
            if st == f.FQA_OK:
                assert torch.equal(out, want), (rank, stage)
            else:
                gave_up += 1
                assert stage < 1 << 24
            if rank <= 0 and stage == 0:
                assert st == f.FQA_ERR_TIMEOUT
            assert (held[M * N:] == -77.0).all()
            # and the next call is what it always is
            assert torch.equal(f.mx_matmul(a, b, out_dtype=1), want), (rank, stage)
            assert f.fqa_debug_status()[0] == f.FQA_OK
    assert gave_up >= 6                     # from stages 0 and 1 on, of every CTA, the first and the second


def test_a_product_that_gave_up_between_others():
    """In a stream with calls before and behind it, nothing waited for: they give
    what they give."""
    f = fqa()
    for M, N in ((1, 1024), (2000, 2048)):
        a, b = R.random_microscaled(M, 4096, "nvfp4", 1), R.random_microscaled(N, 4096, "nvfp4", 2)
        want, out = f.mx_matmul(a, b), torch.empty(M, N, device="cuda")
        torch.cuda.synchronize()
        for rank in (-1, 1):
            before = f.mx_matmul(a, b)
            f.fqa_debug_mx_matmul_timeout(a, b, out, 1, rank, 1)
            behind = [f.mx_matmul(a, b) for _ in range(3)]
            assert f.fqa_debug_status()[0] == f.FQA_ERR_TIMEOUT
            assert all(torch.equal(y, want) for y in (before, *behind))
            assert f.fqa_debug_status()[0] == f.FQA_OK
