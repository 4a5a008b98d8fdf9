"""A launch that the runtime refuses answers FQA_ERR_CUDA, and leaves nothing
behind for the calls that follow.  The refusal comes from a stream whose capture
was ended by a call that capture does not allow: nothing reaches the GPU."""

import contextlib
import ctypes

import pytest
import torch

from tests import block_ref as R

pytestmark = pytest.mark.gpu

ERR_CUDA = 4


@contextlib.contextmanager
def refusing_stream():
    rt = ctypes.CDLL("libcudart.so.12")
    s = torch.cuda.Stream()
    h = ctypes.c_void_p(s.cuda_stream)
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(h, 2) == 0                # 2: relaxed
    assert rt.cudaStreamSynchronize(h) != 0                    # not allowed there: the capture is void
    try:
        yield s
    finally:
        graph = ctypes.c_void_p()
        assert rt.cudaStreamEndCapture(h, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()                                  # this test's own two errors


def calls():
    import quantized_fp8_attention_b200 as f
    L = f.lib()
    x = torch.randn(3, 256, device="cuda").bfloat16()
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    q = f.mx_quantize(x, "nvfp4")
    h = torch.empty_like(x)
    p = lambda t: t.data_ptr()
    large = R.random_microscaled(1500, 64, "mxfp8", 1), R.random_microscaled(2048, 64, "mxfp8", 2)
    y, y1 = torch.empty(1500, 2048, device="cuda"), torch.empty(3, 3, device="cuda")
    r = torch.randn(1, 2, 5, 128, device="cuda").bfloat16()
    ro, pos, axes = torch.empty_like(r), torch.zeros(5, 1, dtype=torch.int32, device="cuda"), (ctypes.c_int * 1)(128)
    a = torch.randn(1, 1, 256, 128, device="cuda").bfloat16()
    qz = f.quantize(a, a, a)
    ao = torch.empty_like(a)
    ws = torch.empty(f.fqa_quantize_workspace_bytes(1, 1, 256), dtype=torch.uint8, device="cuda")
    keep = (x, w, q, h, large, y, y1, r, ro, pos, axes, a, qz, ao, ws)
    at = lambda s: ctypes.c_void_p(s.cuda_stream)
    return keep, {
        "rows": lambda s: L.fqa_mx_quantize(p(x), 0, 3, 256, 256, 2, p(q.codes), p(q.scales), p(q.row_scale), at(s)),
        "rows off": lambda s: L.fqa_mx_quantize(p(x) + 2, 0, 2, 255, 256, 2, p(q.codes), p(q.scales), p(q.row_scale), at(s)),
        "norm": lambda s: L.fqa_mx_rms_norm(p(x), 0, 3, 256, 256, p(w), 0, 1e-6, p(x), 0, 256, 2, p(q.codes),
                                            p(q.scales), p(q.row_scale), p(h), at(s)),
        "back": lambda s: L.fqa_mx_dequantize(p(q.codes), p(q.scales), p(q.row_scale), 3, 256, 2, p(h), 0, at(s)),
        "few rows": lambda s: L.fqa_mx_matmul(p(q.codes), p(q.scales), p(q.row_scale), p(q.codes), p(q.scales),
                                              p(q.row_scale), None, 3, 3, 256, 2, p(y1), 1, at(s)),
        "many rows": lambda s: L.fqa_mx_matmul(p(large[0].codes), p(large[0].scales), None, p(large[1].codes),
                                               p(large[1].scales), None, None, 1500, 2048, 64, 0, p(y), 1, at(s)),
        "rotary": lambda s: L.fqa_rotary(p(r), None, 0, 1, 2, 0, 5, 128, 1280, 640, 128, 0, 0, 0, p(pos), 3, 0, 1, axes,
                                         1e4, 0, None, None, 1e-6, p(ro), None, at(s)),
        "quantize": lambda s: f.fqa_quantize(a, a, a, *qz[:8], ws, stream=s),
        "fp8 attention": lambda s: f.fqa_attention_fp8(*qz[:7], f.softmax_scale(), ao, 0, stream=s),
        "bf16 attention": lambda s: f.fqa_attention_bf16(a, a, a, f.softmax_scale(), ao, 0, stream=s),
    }


def test_a_refused_launch_leaves_no_error_behind():
    keep, table = calls()
    here = torch.cuda.current_stream()
    for name, call in table.items():
        assert call(here) == 0, name
    torch.cuda.synchronize()
    for name, call in table.items():
        with refusing_stream() as s:
            assert call(s) == ERR_CUDA, name
            # the next call is clean, whichever it is, and so is torch's
            for other, again in table.items():
                assert again(here) == 0, (name, other)
        assert float(torch.ones(8, device="cuda").sum()) == 8.0
    torch.cuda.synchronize()
