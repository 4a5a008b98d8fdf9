"""Calls in a row over the same buffers, nothing waited for: every launch of the
operators around the attention begins while the one before it still runs, and
has to give what it gives alone."""

import pytest
import torch

from tests import block_ref as R

pytestmark = pytest.mark.gpu


def fqa():
    import quantized_fp8_attention_b200 as f
    return f


class Chain:
    """Norm, product, rotation of the product's view, quantization, the way back,
    quantization of that into the same buffers, the way back again, product; the
    result is the next round's input."""

    def __init__(self, M, fmt, H=8, K=1024):
        f = fqa()
        g = torch.Generator(device="cuda").manual_seed(M)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.M, self.fmt, self.H, self.K, N = M, fmt, H, K, H * 128
        self.x = rand(M, K).bfloat16()
        self.w = (1 + 0.1 * rand(K)).bfloat16()
        self.up = f.mx_quantize((rand(N, K) / K ** 0.5).bfloat16(), fmt)
        self.down = f.mx_quantize((rand(K, N) / N ** 0.5).bfloat16(), fmt)
        self.bias = rand(K)
        self.rot = f.Rotary(torch.arange(M, dtype=torch.int32, device="cuda")[:, None], (128,),
                            q_weight=torch.ones(128, dtype=torch.bfloat16, device="cuda"))
        self.h, self.step = torch.empty_like(self.x), torch.empty_like(self.x)
        self.q, self.m = f.alloc_microscaled(M, K, fmt, "cuda"), f.alloc_microscaled(M, N, fmt, "cuda")
        self.mid = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        self.turned = torch.empty(1, H, M, 128, dtype=torch.bfloat16, device="cuda")
        self.v, self.v2 = torch.empty_like(self.mid), torch.empty_like(self.mid)

    def reset(self):
        self.h.zero_()
        self.step.copy_(self.x)

    def round(self, after):
        f = fqa()
        f.mx_rms_norm(self.step, self.w, self.fmt, residual=self.h, residual_out=self.h, out=self.q)
        after()
        f.mx_matmul(self.q, self.up, out=self.mid)
        after()
        f.rotary(self.mid.view(1, self.M, self.H, 128).transpose(1, 2), None, self.rot, q_out=self.turned)
        after()
        f.mx_quantize(self.turned.view(self.M, -1), self.fmt, out=self.m)
        after()
        f.mx_dequantize(self.m, out=self.v)
        after()
        f.mx_quantize(self.v, self.fmt, out=self.m)
        after()
        f.mx_dequantize(self.m, out=self.v2)
        after()
        f.mx_matmul(self.m, self.down, bias=self.bias, out=self.step)
        after()

    def state(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.h, self.step, self.v, self.v2, self.mid, self.turned)]


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("M", [1, 40, 500, 3000])     # clusters, wider tiles, one CTA a tile, pairs of CTAs
def test_the_whole_chain(M, fmt):
    f = fqa()
    c, rounds = Chain(M, fmt), 12
    c.reset()
    for _ in range(rounds):
        c.round(torch.cuda.synchronize)
    want = c.state()
    assert all(torch.isfinite(t).all() for t in want)
    c.reset()
    for _ in range(rounds):
        c.round(lambda: None)
    assert all(torch.equal(a, b) for a, b in zip(want, c.state()))
    # replayed, the launches follow one another without the host between them
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(rounds):
            c.round(lambda: None)
    for _ in range(20):
        c.reset()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, c.state()))
    assert f.fqa_debug_status()[0] == f.FQA_OK


@pytest.mark.parametrize("M", [4, 1500])
def test_codes_and_row_scales_written_again_and_again(M):
    """The way back, new rows into the same buffers, the way back: some hundred
    times in a graph, each result kept.  The row scales differ from round to
    round by powers of two, so a row scale of the round before shows."""
    f = fqa()
    rounds = 200
    x = torch.randn(rounds, M, 320, device="cuda") * 2.0 ** (torch.arange(rounds, device="cuda") % 37)[:, None, None]
    w = torch.ones(320, device="cuda")
    b = R.random_microscaled(2048 if M > 64 else 256, 320, "nvfp4", 5, wide=True)
    want = [f.mx_dequantize(f.mx_quantize(t, "nvfp4")) for t in x]
    wanty = [f.mx_matmul(f.mx_quantize(t, "nvfp4"), b) for t in x]
    wantn = [f.mx_matmul(f.mx_rms_norm(t, w, "nvfp4", eps=0.0)[0], b) for t in x]
    torch.cuda.synchronize()
    q = f.alloc_microscaled(M, 320, "nvfp4", "cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = []
        for t in x:
            f.mx_quantize(t, "nvfp4", out=q)
            got.append((f.mx_dequantize(q), f.mx_matmul(q, b)))
            f.mx_rms_norm(t, w, "nvfp4", eps=0.0, out=q)
            got[-1] += (f.mx_matmul(q, b),)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        for i in range(rounds):
            assert torch.equal(got[i][0], want[i]) and torch.equal(got[i][1], wanty[i]) and torch.equal(got[i][2], wantn[i])
    assert f.fqa_debug_status()[0] == f.FQA_OK
