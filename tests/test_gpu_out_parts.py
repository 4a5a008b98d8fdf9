"""Outputs whose own parts share memory are refused."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_codes_scales_and_row_scales_lie_apart(fmt):
    import quantized_fp8_attention_b200 as f
    x = torch.randn(128, 256, device="cuda")
    w = torch.ones(256, device="cuda")
    good = f.alloc_microscaled(128, 256, fmt, "cuda")
    n, m = good.codes.numel(), good.scales.numel()
    held = torch.empty(n + m + 512, dtype=torch.uint8, device="cuda")
    codes = held[:n].view(good.codes.shape)
    apart = good._replace(codes=codes, scales=held[n: n + m].view(good.scales.shape))
    bad = [good._replace(codes=codes, scales=held[n - 16: n - 16 + m].view(good.scales.shape))]
    if fmt == "nvfp4":
        apart = apart._replace(row_scale=held[n + m:].view(torch.float32))
        bad.append(good._replace(codes=codes, row_scale=held[n - 512: n].view(torch.float32)))
        bad.append(apart._replace(row_scale=held[n + m - 4: n + m + 508].view(torch.float32)))
    for out in bad:
        for call in (lambda: f.mx_quantize(x, fmt, out=out), lambda: f.mx_rms_norm(x, w, fmt, out=out)):
            with pytest.raises(ValueError, match="overlaps"):
                call()
    want = f.mx_dequantize(f.mx_quantize(x, fmt))
    assert torch.equal(f.mx_dequantize(f.mx_quantize(x, fmt, out=apart)), want)
