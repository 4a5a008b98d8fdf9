"""Captured work that forks and joins around the overlapped launches."""

import pytest
import torch

from tests import block_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("M", [3, 300, 2000])
def test_two_branches_join_in_a_product(M, fmt):
    """Rows and weights quantized on streams of their own, joined by events, then
    products on both streams, the way back, a copy and a norm: replayed on inputs
    that change, equal to the same calls one at a time."""
    import quantized_fp8_attention_b200 as f
    K, N = 512, 2048
    g = torch.Generator(device="cuda").manual_seed(M)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    x, w, norm = rand(M, K), rand(N, K), rand(K)

    def serial():
        a, b = f.mx_quantize(x, fmt), f.mx_quantize(w, fmt)
        y = f.mx_matmul(a, b, out_dtype=1)
        n, _ = f.mx_rms_norm(f.mx_dequantize(a, 1), norm, fmt)
        return y, f.mx_matmul(n, b, out_dtype=1)

    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    for t in (*serial(), x, w):
        t.record_stream(main)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            b = f.mx_quantize(w, fmt)
        a = f.mx_quantize(x, fmt)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            back = f.mx_dequantize(a, 1).clone()
            n, _ = f.mx_rms_norm(back, norm, fmt)
        main.wait_stream(side)
        y = f.mx_matmul(a, b, out_dtype=1)
        z = f.mx_matmul(n, b, out_dtype=1)
    for _ in range(4):
        x.copy_(rand(M, K))
        w.copy_(rand(N, K))
        want = serial()
        torch.cuda.synchronize()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])
    assert f.fqa_debug_status()[0] == f.FQA_OK
