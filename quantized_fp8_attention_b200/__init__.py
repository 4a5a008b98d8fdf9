"""Python binding of libfqa.so, the B200 FP8 quantized attention library.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch provides device memory and the current stream.  The C ABI
is declared (and documented) in include/fqa.h; the functions below carry the
same names and pass ``tensor.data_ptr()`` and the stream handle through.

The library must have been built (``python -m quantized_fp8_attention_b200.build``
or ``__graft_entry__.build()``); every call raises ImportError without it.
"""

from __future__ import annotations

import ctypes
import functools
import operator
import os
import warnings
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfqa.so")

FQA_OK, FQA_ERR_INVALID_ARG, FQA_ERR_UNSUPPORTED, FQA_ERR_MISALIGNED, FQA_ERR_CUDA, FQA_ERR_TIMEOUT = range(6)
FQA_OUT_BF16, FQA_OUT_F32 = 0, 1
FQA_OUT_F16 = 2            # mx_matmul and mx_dequantize only: the attention calls refuse it
HEAD_DIM = 128

_lib = None
_native = None             # csrc/binding.cpp: the everyday calls without the interpreter (or _CheckedWay)


def _load():
    """Load libfqa.so and declare the C signatures.  Raises if it is not built:
    there is no fallback implementation."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libfqa.so is not built ({LIB_PATH}); run `python -m quantized_fp8_attention_b200.build`. "
            "There is no fallback implementation.")
    L = ctypes.CDLL(LIB_PATH)
    P, I = ctypes.c_void_p, ctypes.c_int
    L.fqa_version.restype = I
    L.fqa_status_string.restype = ctypes.c_char_p
    L.fqa_status_string.argtypes = [I]
    L.fqa_quantize_workspace_bytes.restype = ctypes.c_size_t
    L.fqa_quantize_workspace_bytes.argtypes = [I, I, I, I]
    L.fqa_quantize.restype = I
    L.fqa_quantize.argtypes = [P, P, P, I, I, I, I, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.fqa_attention_fp8.restype = I
    L.fqa_attention_fp8.argtypes = [P, P, P, P, P, P, P, I, I, I, I, ctypes.c_float, P, I, P]
    L.fqa_attention_bf16.restype = I
    L.fqa_attention_bf16.argtypes = [P, P, P, I, I, I, I, ctypes.c_float, P, I, P]
    L.fqa_e4m3_encode.restype = I
    L.fqa_e4m3_encode.argtypes = [P, P, ctypes.c_size_t, P]
    L.fqa_debug_status.restype = I
    L.fqa_debug_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
    L.fqa_quantize_a2a.restype = I
    L.fqa_quantize_a2a.argtypes = [P, P, P, I, I, I, I, I, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.fqa_attention_fp8_a2a.restype = I
    L.fqa_attention_fp8_a2a.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, ctypes.c_float, P, I, P]
    L.fqa_quantize_keyerr.restype = I
    L.fqa_quantize_keyerr.argtypes = [P, P, P, I, I, I, I, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.fqa_corrected_keys.restype = I
    L.fqa_corrected_keys.argtypes = [I, ctypes.c_float]
    L.fqa_select_keys.restype = I
    L.fqa_select_keys.argtypes = [P, I, I, I, I, P, P, P]
    L.fqa_attention_fp8_corrected_workspace_bytes.restype = ctypes.c_size_t
    L.fqa_attention_fp8_corrected_workspace_bytes.argtypes = [I, I, I, I, ctypes.c_float]
    L.fqa_attention_fp8_corrected.restype = I
    L.fqa_attention_fp8_corrected.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, ctypes.c_float,
                                              ctypes.c_float, P, I, P, ctypes.c_size_t, P]
    L.fqa_quantize_nvfp4_qk.restype = I
    L.fqa_quantize_nvfp4_qk.argtypes = [P, P, P, I, I, I, I, P, P, P, P, P, P, P]
    L.fqa_attention_nvfp4.restype = I
    L.fqa_attention_nvfp4.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, ctypes.c_float, P, I, P]
    L.fqa_e2m1_encode.restype = I
    L.fqa_e2m1_encode.argtypes = [P, P, ctypes.c_size_t, P]
    L.fqa_exp2_error.restype = I
    L.fqa_exp2_error.argtypes = [ctypes.c_float, ctypes.c_float, P, P]
    Z, Q = ctypes.c_size_t, ctypes.c_int64
    for f in (L.fqa_mx_code_bytes, L.fqa_mx_scale_bytes):
        f.restype = Z
        f.argtypes = [I, I, I]
    L.fqa_mx_quantize.restype = I
    L.fqa_mx_quantize.argtypes = [P, I, I, I, Q, I, P, P, P, P]
    L.fqa_mx_rms_norm.restype = I
    L.fqa_mx_rms_norm.argtypes = [P, I, I, I, Q, P, I, ctypes.c_float, P, I, Q, I, P, P, P, P, P]
    L.fqa_mx_dequantize.restype = I
    L.fqa_mx_dequantize.argtypes = [P, P, P, I, I, I, P, I, P]
    L.fqa_mx_matmul.restype = I
    L.fqa_mx_matmul.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P, I, P]
    L.fqa_rotary.restype = I
    L.fqa_rotary.argtypes = [P, P, I, I, I, I, I, I, Q, Q, Q, Q, Q, Q, P, I, Q, I, P, ctypes.c_double, I, P, P,
                             ctypes.c_float, P, P, P]
    global _native
    _native = _short_way()
    _lib = L
    return L


class _CheckedWay:
    """Stands in for csrc/binding.cpp where that is not built for this torch and
    Python: answers None, so every call takes the functions below, 10 to 15 us
    slower on the host."""

    @staticmethod
    def quantize(*args):
        return None

    dequantize = rms_norm = matmul = rotate = quantize


def _short_way():
    from . import build
    try:
        if not build.binding_fits():
            raise ImportError("it is absent or built for another torch or Python")
        from . import _binding
        _binding.init(LIB_PATH, Microscaled, Rotary)
        return _binding
    except ImportError as e:
        warnings.warn(f"_binding.so does not serve ({e}): calls take the slower way through Python; run "
                      "`python -m quantized_fp8_attention_b200.build`.", RuntimeWarning, stacklevel=4)
        return _CheckedWay


def _native_calls():
    _load()
    return _native


class FqaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def lib():
    """The loaded ctypes library (for tests that call the ABI directly)."""
    return _load()


def status_string(status: int) -> str:
    return _load().fqa_status_string(int(status)).decode()


def version() -> int:
    return _load().fqa_version()


def _check(status: int, where: str):
    if status != FQA_OK:
        raise FqaError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ------------------------------------------------------------- raw ABI

def fqa_quantize_workspace_bytes(B: int, H: int, N: int, d: int = HEAD_DIM) -> int:
    return int(_load().fqa_quantize_workspace_bytes(B, H, N, d))


def fqa_quantize(q, k, v, q8, k8, v8, sq, sk, sv, sv_max, k_mean, workspace, stream=None) -> int:
    """The C call with tensors; returns the fqa_status code."""
    B, H, N, d = q.shape
    return _load().fqa_quantize(_ptr(q), _ptr(k), _ptr(v), B, H, N, d, _ptr(q8), _ptr(k8), _ptr(v8),
                             _ptr(sq), _ptr(sk), _ptr(sv), _ptr(sv_max), _ptr(k_mean),
                             _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream(stream))


def fqa_quantize_noalloc(q, k, v, q8, k8, v8, sq, sk, sv, sv_max, k_mean, stream=None) -> int:
    """fqa_quantize without a workspace (for callers that cannot allocate
    device memory when they call): the library keeps the scratch in a fixed
    8 MiB array per GPU.  Returns the fqa_status code."""
    L = _load()
    f = L.fqa_quantize_noalloc
    P, I = ctypes.c_void_p, ctypes.c_int
    f.restype = I
    f.argtypes = [P, P, P, I, I, I, I, P, P, P, P, P, P, P, P, P]
    B, H, N, d = q.shape
    return f(_ptr(q), _ptr(k), _ptr(v), B, H, N, d, _ptr(q8), _ptr(k8), _ptr(v8), _ptr(sq),
             _ptr(sk), _ptr(sv), _ptr(sv_max), _ptr(k_mean), _stream(stream))


def fqa_attention_fp8(q8, k8, v8, sq, sk, sv, sv_max, softmax_scale, out, out_dtype, stream=None) -> int:
    B, H, N, d = q8.shape
    return _load().fqa_attention_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(sq), _ptr(sk), _ptr(sv),
                                  _ptr(sv_max), B, H, N, d, float(softmax_scale), _ptr(out),
                                  int(out_dtype), _stream(stream))


def fqa_attention_bf16(q, k, v, softmax_scale, out, out_dtype, stream=None) -> int:
    B, H, N, d = q.shape
    return _load().fqa_attention_bf16(_ptr(q), _ptr(k), _ptr(v), B, H, N, d, float(softmax_scale),
                                   _ptr(out), int(out_dtype), _stream(stream))


def fqa_quantize_a2a(q, k, v, q8, k8, v8, sq, sk, sv, sv_max, k_mean, workspace, stream=None) -> int:
    """fqa_quantize on inputs in the sequence all-to-all layout [B, P, Hl, Nl, d]."""
    B, P, Hl, Nl, d = q.shape
    return _load().fqa_quantize_a2a(_ptr(q), _ptr(k), _ptr(v), B, Hl, P, Nl, d, _ptr(q8), _ptr(k8), _ptr(v8),
                                 _ptr(sq), _ptr(sk), _ptr(sv), _ptr(sv_max), _ptr(k_mean), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream))


def fqa_attention_fp8_a2a(q8, k8, v8, sq, sk, sv, sv_max, P: int, softmax_scale, out, out_dtype,
                          stream=None) -> int:
    """fqa_attention_fp8 writing out in the layout [B, P, Hl, N / P, d]."""
    B, Hl, N, d = q8.shape
    return _load().fqa_attention_fp8_a2a(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(sq), _ptr(sk), _ptr(sv),
                                      _ptr(sv_max), B, Hl, int(P), N // int(P), d, float(softmax_scale),
                                      _ptr(out), int(out_dtype), _stream(stream))


def fqa_quantize_keyerr(q, k, v, q8, k8, v8, sq, sk, sv, sv_max, k_mean, k_err, workspace,
                        stream=None) -> int:
    """fqa_quantize plus each key's quantization error k_err [B,H,N] FP32."""
    B, H, N, d = q.shape
    return _load().fqa_quantize_keyerr(_ptr(q), _ptr(k), _ptr(v), B, H, N, d, _ptr(q8), _ptr(k8), _ptr(v8),
                                    _ptr(sq), _ptr(sk), _ptr(sv), _ptr(sv_max), _ptr(k_mean), _ptr(k_err),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream))


def fqa_corrected_keys(N: int, rho: float) -> int:
    return int(_load().fqa_corrected_keys(int(N), float(rho)))


def fqa_select_keys(k_err, kc: int, kmask, idx, stream=None) -> int:
    B, H, N = k_err.shape
    return _load().fqa_select_keys(_ptr(k_err), B, H, N, int(kc), _ptr(kmask), _ptr(idx), _stream(stream))


def fqa_attention_fp8_corrected_workspace_bytes(B: int, H: int, N: int, rho: float, d: int = HEAD_DIM) -> int:
    return int(_load().fqa_attention_fp8_corrected_workspace_bytes(B, H, N, d, float(rho)))


def fqa_attention_fp8_corrected(q, k, v, q8, k8, v8, sq, sk, sv, sv_max, k_mean, k_err, softmax_scale, rho,
                                out, out_dtype, workspace, stream=None) -> int:
    B, H, N, d = q.shape
    return _load().fqa_attention_fp8_corrected(
        _ptr(q), _ptr(k), _ptr(v), _ptr(q8), _ptr(k8), _ptr(v8), _ptr(sq), _ptr(sk), _ptr(sv), _ptr(sv_max),
        _ptr(k_mean), _ptr(k_err), B, H, N, d, float(softmax_scale), float(rho), _ptr(out), int(out_dtype),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))


def fqa_e4m3_encode(x, out, stream=None) -> int:
    return _load().fqa_e4m3_encode(_ptr(x), _ptr(out), x.numel(), _stream(stream))


def fqa_quantize_nvfp4_qk(q, k, k_mean, q4, k4, sfq, sfk, sq1, sk1, stream=None) -> int:
    B, H, N, d = q.shape
    return _load().fqa_quantize_nvfp4_qk(_ptr(q), _ptr(k), _ptr(k_mean), B, H, N, d, _ptr(q4), _ptr(k4),
                                         _ptr(sfq), _ptr(sfk), _ptr(sq1), _ptr(sk1), _stream(stream))


def fqa_attention_nvfp4(q4, k4, sfq, sfk, sq1, sk1, v8, sv, sv_max, softmax_scale, out, out_dtype,
                        stream=None) -> int:
    B, H, N, d = v8.shape
    return _load().fqa_attention_nvfp4(_ptr(q4), _ptr(k4), _ptr(sfq), _ptr(sfk), _ptr(sq1), _ptr(sk1), _ptr(v8),
                                       _ptr(sv), _ptr(sv_max), B, H, N, d, float(softmax_scale), _ptr(out),
                                       int(out_dtype), _stream(stream))


def fqa_e2m1_encode(x, out, stream=None) -> int:
    return _load().fqa_e2m1_encode(_ptr(x), _ptr(out), x.numel() // 2, _stream(stream))


def fqa_exp2_error(lo: float, hi: float, max_rel_bits, stream=None) -> int:
    return _load().fqa_exp2_error(float(lo), float(hi), _ptr(max_rel_bits), _stream(stream))


def exp2_max_rel_error(lo: float, hi: float, device="cuda") -> float:
    """Largest relative error of the kernels' exp2 over every binary32 in [lo, hi]."""
    bits = torch.zeros(1, dtype=torch.int32, device=device)
    _check(fqa_exp2_error(lo, hi, bits), "fqa_exp2_error")
    return float(bits.cpu().view(torch.float32)[0])


def fqa_debug_wait_timeout(limit_us: int, stream=None) -> int:
    """Launch a bounded wait that is bound to give up after limit_us (tests the
    timeout path; the next fqa_debug_status() reports FQA_ERR_TIMEOUT)."""
    L = _load()
    L.fqa_debug_wait_timeout.restype = ctypes.c_int
    L.fqa_debug_wait_timeout.argtypes = [ctypes.c_uint32, ctypes.c_void_p]
    return L.fqa_debug_wait_timeout(int(limit_us), _stream(stream))


def fqa_debug_mx_matmul_timeout(a: "Microscaled", b: "Microscaled", out: torch.Tensor, out_dtype: int, rank: int = -1,
                                stage: int = 0, stream=None) -> int:
    """mx_matmul(a, b) into out with loads that stop at a stage and waits that
    give up early (the next fqa_debug_status() reports FQA_ERR_TIMEOUT)."""
    L = _load()
    P, I = ctypes.c_void_p, ctypes.c_int
    L.fqa_debug_mx_matmul_timeout.restype = I
    L.fqa_debug_mx_matmul_timeout.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P, I, I, I, P]
    M, code, index = _require_microscaled(a, "a")
    N, other, _ = _require_microscaled(b, "b", index)
    if other != code or a.cols != b.cols:
        raise ValueError(f"a and b: {a.fmt} rows of {a.cols} against {b.fmt} rows of {b.cols}")
    _device_tensor(out, "out", index)
    _require(out, _OUT_DTYPE[out_dtype], "out", (M, N))
    return L.fqa_debug_mx_matmul_timeout(_ptr(a.codes), _ptr(a.scales), _ptr(a.row_scale), _ptr(b.codes), _ptr(b.scales),
                                         _ptr(b.row_scale), None, M, N, a.cols, code, _ptr(out), int(out_dtype),
                                         int(rank), int(stage), _stream(stream))


def fqa_debug_status(stream=None):
    """(status, raw flag bits) of the current device's status word; clears it."""
    flags = ctypes.c_uint32(0)
    st = _load().fqa_debug_status(_stream(stream), ctypes.byref(flags))
    return st, flags.value


# ----------------------------------------------------- tensor-level API

def _require(t, dtype: torch.dtype, name: str, shape=None) -> None:
    """The C ABI takes contiguous device buffers of a fixed element type and
    shape; anything else is refused here, before a pointer is passed on."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _require_qkv(q, k, v, dtype: torch.dtype):
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q: expected a [B, H, N, 128] tensor")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require(t, dtype, name, q.shape)
    if q.device != k.device or q.device != v.device:
        raise ValueError("q, k and v must be on the same device")
    return tuple(q.shape)


def nblocks(N: int) -> int:
    """64-token blocks per head: ceil(N / 64) (the last one may be short)."""
    return (N + 63) // 64


def _require_quantized(qz: "Quantized", B: int, H: int, N: int) -> None:
    nb = nblocks(N)
    shapes = ((B, H, N, HEAD_DIM),) * 3 + ((B, H, nb),) * 3 + ((B, H), (B, H, HEAD_DIM))
    for name, t, shape in zip(Quantized._fields, qz, shapes):
        _require(t, torch.uint8 if name.endswith("8") else torch.float32, name, shape)


class Quantized(NamedTuple):
    q8: torch.Tensor       # uint8 E4M3 codes [B,H,N,128]
    k8: torch.Tensor
    v8: torch.Tensor
    sq: torch.Tensor       # float32 [B,H,ceil(N/64)]
    sk: torch.Tensor
    sv: torch.Tensor
    sv_max: torch.Tensor   # float32 [B,H]
    k_mean: torch.Tensor   # float32 [B,H,128]


def alloc_quantized(B: int, H: int, N: int, device) -> Quantized:
    u8 = dict(dtype=torch.uint8, device=device)
    f32 = dict(dtype=torch.float32, device=device)
    nb = nblocks(N)
    return Quantized(torch.empty(B, H, N, HEAD_DIM, **u8), torch.empty(B, H, N, HEAD_DIM, **u8),
                     torch.empty(B, H, N, HEAD_DIM, **u8), torch.empty(B, H, nb, **f32),
                     torch.empty(B, H, nb, **f32), torch.empty(B, H, nb, **f32),
                     torch.empty(B, H, **f32), torch.empty(B, H, HEAD_DIM, **f32))


def alloc_workspace(B: int, H: int, N: int, device) -> torch.Tensor:
    nbytes = fqa_quantize_workspace_bytes(B, H, N)
    return torch.empty(max(nbytes, 16) // 4, dtype=torch.float32, device=device)


def quantize(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: Optional[Quantized] = None,
             workspace: Optional[torch.Tensor] = None, stream=None) -> Quantized:
    """BF16 [B,H,N,128] Q, K, V (CUDA, contiguous) -> Quantized."""
    B, H, N, _ = _require_qkv(q, k, v, torch.bfloat16)
    if out is None:
        out = alloc_quantized(B, H, N, q.device)
    _require_quantized(out, B, H, N)
    if workspace is None:
        workspace = alloc_workspace(B, H, N, q.device)
    _require(workspace, workspace.dtype, "workspace")
    _check(fqa_quantize(q, k, v, *out, workspace, stream=stream), "fqa_quantize")
    return out


def attention_fp8(qz: Quantized, softmax_scale: float, out_dtype: int = FQA_OUT_BF16,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    if not isinstance(qz.q8, torch.Tensor) or qz.q8.dim() != 4:
        raise ValueError("qz.q8: expected a [B, H, N, 128] tensor")
    B, H, N, d = qz.q8.shape
    _require_quantized(qz, B, H, N)
    dt = torch.float32 if out_dtype == FQA_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty(B, H, N, d, dtype=dt, device=qz.q8.device)
    _require(out, dt, "out", (B, H, N, d))
    _check(fqa_attention_fp8(qz.q8, qz.k8, qz.v8, qz.sq, qz.sk, qz.sv, qz.sv_max, softmax_scale,
                             out, out_dtype, stream=stream), "fqa_attention_fp8")
    return out


def attention_bf16(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, softmax_scale: float,
                   out_dtype: int = FQA_OUT_BF16, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    B, H, N, d = _require_qkv(q, k, v, torch.bfloat16)
    dt = torch.float32 if out_dtype == FQA_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty(B, H, N, d, dtype=dt, device=q.device)
    _require(out, dt, "out", (B, H, N, d))
    _check(fqa_attention_bf16(q, k, v, softmax_scale, out, out_dtype, stream=stream),
           "fqa_attention_bf16")
    return out


def quantize_keyerr(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: Optional[Quantized] = None,
                    k_err: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None):
    """quantize() plus the per-key quantization error: (Quantized, k_err [B,H,N] float32)."""
    B, H, N, _ = _require_qkv(q, k, v, torch.bfloat16)
    if out is None:
        out = alloc_quantized(B, H, N, q.device)
    _require_quantized(out, B, H, N)
    if k_err is None:
        k_err = torch.empty(B, H, N, dtype=torch.float32, device=q.device)
    _require(k_err, torch.float32, "k_err", (B, H, N))
    if workspace is None:
        workspace = alloc_workspace(B, H, N, q.device)
    _require(workspace, workspace.dtype, "workspace")
    _check(fqa_quantize_keyerr(q, k, v, *out, k_err, workspace, stream=stream), "fqa_quantize_keyerr")
    return out, k_err


def quantize_a2a(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: Optional[Quantized] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> Quantized:
    """Q, K, V in the sequence all-to-all layout [B, P, Hl, Nl, 128] (BF16,
    CUDA, contiguous; Nl a multiple of 64) -> Quantized for B, Hl heads and
    N = P * Nl tokens in the usual layouts."""
    if not isinstance(q, torch.Tensor) or q.dim() != 5:
        raise ValueError("q: expected a [B, P, Hl, Nl, 128] tensor")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require(t, torch.bfloat16, name, q.shape)
    B, P, Hl, Nl, _ = q.shape
    N = P * Nl
    if out is None:
        out = alloc_quantized(B, Hl, N, q.device)
    _require_quantized(out, B, Hl, N)
    if workspace is None:
        workspace = alloc_workspace(B, Hl, N, q.device)
    _require(workspace, workspace.dtype, "workspace")
    _check(fqa_quantize_a2a(q, k, v, *out, workspace, stream=stream), "fqa_quantize_a2a")
    return out


def attention_fp8_a2a(qz: Quantized, P: int, softmax_scale: float, out_dtype: int = FQA_OUT_BF16,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fqa_attention_fp8 with the output in the layout [B, P, Hl, N / P, 128]."""
    B, Hl, N, d = qz.q8.shape
    _require_quantized(qz, B, Hl, N)
    if N % P:
        raise ValueError(f"N = {N} is not a multiple of P = {P}")
    dt = torch.float32 if out_dtype == FQA_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty(B, P, Hl, N // P, d, dtype=dt, device=qz.q8.device)
    _require(out, dt, "out", (B, P, Hl, N // P, d))
    _check(fqa_attention_fp8_a2a(*qz[:7], P, softmax_scale, out, out_dtype, stream=stream),
           "fqa_attention_fp8_a2a")
    return out


def alloc_corrected_workspace(B: int, H: int, N: int, rho: float, device) -> torch.Tensor:
    nbytes = fqa_attention_fp8_corrected_workspace_bytes(B, H, N, rho)
    if nbytes == 0:
        raise ValueError("invalid sizes or rho for the corrected path")
    return torch.empty((nbytes + 15) // 16 * 4, dtype=torch.float32, device=device)


def attention_fp8_corrected(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, qz: Quantized,
                            k_err: torch.Tensor, softmax_scale: float, rho: float = 0.005,
                            out_dtype: int = FQA_OUT_BF16, out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Error-corrected FP8 attention: the ceil(rho * N) keys per head with the
    largest quantization error are handled exactly, the rest by the FP8 rule."""
    B, H, N, d = _require_qkv(q, k, v, torch.bfloat16)
    _require_quantized(qz, B, H, N)
    _require(k_err, torch.float32, "k_err", (B, H, N))
    dt = torch.float32 if out_dtype == FQA_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty(B, H, N, d, dtype=dt, device=q.device)
    _require(out, dt, "out", (B, H, N, d))
    if workspace is None:
        workspace = alloc_corrected_workspace(B, H, N, rho, q.device)
    _require(workspace, workspace.dtype, "workspace")
    _check(fqa_attention_fp8_corrected(q, k, v, *qz[:7], qz.k_mean, k_err, softmax_scale, rho, out, out_dtype,
                                       workspace, stream=stream), "fqa_attention_fp8_corrected")
    return out


def fp8_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, softmax_scale: float,
                  out_dtype: int = FQA_OUT_BF16, stream=None, rot: Optional["Rotary"] = None) -> torch.Tensor:
    """The whole FP8 path: with rot, rotary() on q and k (which may then be
    strided views; as many heads as v, which is contiguous); quantize; fused FP8
    attention."""
    if rot is not None:
        q, k = rotary(q, k, rot, stream=stream)
    return attention_fp8(quantize(q, k, v, stream=stream), softmax_scale, out_dtype, stream=stream)


def e4m3_encode(x: torch.Tensor, stream=None) -> torch.Tensor:
    _require(x, torch.float32, "x")
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(fqa_e4m3_encode(x, out, stream=stream), "fqa_e4m3_encode")
    return out


# ------------------------------------------------ NVFP4 Q.K variant

class QuantizedNvfp4(NamedTuple):
    q4: torch.Tensor       # uint8 [B,H,N,64]: E2M1 codes, element 2i in the low nibble
    k4: torch.Tensor       # of K - k_mean
    sfq: torch.Tensor      # uint8 [B,H,N,8]: E4M3 scale per 16 channels
    sfk: torch.Tensor
    sq1: torch.Tensor      # float32 [B,H,ceil(N/64)]
    sk1: torch.Tensor


def alloc_quantized_nvfp4(B: int, H: int, N: int, device) -> QuantizedNvfp4:
    u8 = dict(dtype=torch.uint8, device=device)
    f32 = dict(dtype=torch.float32, device=device)
    nb = nblocks(N)
    return QuantizedNvfp4(torch.empty(B, H, N, HEAD_DIM // 2, **u8), torch.empty(B, H, N, HEAD_DIM // 2, **u8),
                          torch.empty(B, H, N, HEAD_DIM // 16, **u8), torch.empty(B, H, N, HEAD_DIM // 16, **u8),
                          torch.empty(B, H, nb, **f32), torch.empty(B, H, nb, **f32))


def _require_nvfp4(qn: QuantizedNvfp4, B: int, H: int, N: int) -> None:
    nb = nblocks(N)
    shapes = ((B, H, N, HEAD_DIM // 2),) * 2 + ((B, H, N, HEAD_DIM // 16),) * 2 + ((B, H, nb),) * 2
    for name, t, shape in zip(QuantizedNvfp4._fields, qn, shapes):
        _require(t, torch.float32 if name.endswith("1") else torch.uint8, name, shape)


def quantize_nvfp4_qk(q: torch.Tensor, k: torch.Tensor, k_mean: torch.Tensor,
                      out: Optional[QuantizedNvfp4] = None, stream=None) -> QuantizedNvfp4:
    """BF16 Q, K [B,H,N,128] and the K channel means of quantize() -> NVFP4 Q and
    smoothed K."""
    B, H, N, _ = _require_qkv(q, k, k, torch.bfloat16)
    _require(k_mean, torch.float32, "k_mean", (B, H, HEAD_DIM))
    if out is None:
        out = alloc_quantized_nvfp4(B, H, N, q.device)
    _require_nvfp4(out, B, H, N)
    _check(fqa_quantize_nvfp4_qk(q, k, k_mean, *out, stream=stream), "fqa_quantize_nvfp4_qk")
    return out


def attention_nvfp4(qn: QuantizedNvfp4, qz: Quantized, softmax_scale: float, out_dtype: int = FQA_OUT_BF16,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """NVFP4 Q.K^T, FP8 P.V: qn from quantize_nvfp4_qk(), V (v8, sv, sv_max) from qz."""
    if not isinstance(qz.v8, torch.Tensor) or qz.v8.dim() != 4:
        raise ValueError("qz.v8: expected a [B, H, N, 128] tensor")
    B, H, N, d = qz.v8.shape
    _require_quantized(qz, B, H, N)
    _require_nvfp4(qn, B, H, N)
    dt = torch.float32 if out_dtype == FQA_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty(B, H, N, d, dtype=dt, device=qz.v8.device)
    _require(out, dt, "out", (B, H, N, d))
    _check(fqa_attention_nvfp4(*qn, qz.v8, qz.sv, qz.sv_max, softmax_scale, out, out_dtype, stream=stream),
           "fqa_attention_nvfp4")
    return out


def nvfp4_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, softmax_scale: float,
                    out_dtype: int = FQA_OUT_BF16, stream=None, rot: Optional["Rotary"] = None) -> torch.Tensor:
    """The whole FP4 Q.K path: with rot, rotary() on q and k; quantize (V codes
    and the K mean), NVFP4 Q and K, then the attention."""
    if rot is not None:
        q, k = rotary(q, k, rot, stream=stream)
    qz = quantize(q, k, v, stream=stream)
    return attention_nvfp4(quantize_nvfp4_qk(q, k, qz.k_mean, stream=stream), qz, softmax_scale, out_dtype,
                           stream=stream)


def e2m1_encode(x: torch.Tensor, stream=None) -> torch.Tensor:
    """FP32 [..., 2n] -> uint8 [..., n]: two E2M1 codes per byte, x[2i] in the low nibble."""
    _require(x, torch.float32, "x")
    if x.numel() % 2:
        raise ValueError("x: expected an even number of elements")
    out = torch.empty(x.numel() // 2, dtype=torch.uint8, device=x.device)
    _check(fqa_e2m1_encode(x, out, stream=stream), "fqa_e2m1_encode")
    return out


# ------------------------------------- rotary positions, microscaled rows
#
# Each function first tries csrc/binding.cpp, which takes the everyday call: no
# output or stream given, tensors on the current device, eps and theta floats, axes
# a tuple, split, shared and inverse truth values.  Any other call costs 10 to 15 us
# more on the host.

_DTYPE = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2, torch.int32: 3}
_OUT_DTYPE = {FQA_OUT_BF16: torch.bfloat16, FQA_OUT_F32: torch.float32, FQA_OUT_F16: torch.float16}
MX_FORMATS = {"mxfp8": 0, "mxfp4": 1, "nvfp4": 2}
_MX_MAX_ROWS, _MX_MAX_COLS = 1 << 24, 1 << 20


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(index: int, stream, inputs):
    """None where a call is for the current device and stream.  Otherwise the
    context that makes them so: the tensors' device becomes current, and where a
    stream is given outputs are allocated on it and the tensors given marked as
    used by it."""
    if stream is None:
        return None if index == torch.cuda.current_device() else torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    for t in inputs:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _device_tensor(t, name: str, index: int = -1) -> int:
    """The index of a CUDA tensor's device (the one given, if one is)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    got = t.get_device()
    if got < 0 or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    if index >= 0 and got != index:
        raise ValueError(f"{name}: expected a tensor on cuda:{index}, got one on {t.device}")
    return got


def _extent(t: torch.Tensor):
    """First byte and the one past the last that the tensor's elements touch."""
    n = 0 if t.numel() == 0 else sum((s - 1) * st for s, st in zip(t.shape, t.stride())) + 1
    return t.data_ptr(), t.data_ptr() + n * t.element_size()


def _apart(out: torch.Tensor, name: str, inputs) -> None:
    """Refuses an output that shares memory with one of the inputs."""
    lo, hi = _extent(out)
    for t in inputs:
        if t is not None:
            a, b = _extent(t)
            if lo < b and a < hi:
                raise ValueError(f"{name}: overlaps another tensor of the call")


def _same_memory(a: torch.Tensor, b: torch.Tensor) -> bool:
    return a.data_ptr() == b.data_ptr() and a.dtype == b.dtype and a.is_contiguous() and b.is_contiguous()


def _float_dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPE.get(t.dtype, 3)
    if code == 3:
        raise ValueError(f"{name}: expected bfloat16, float16 or float32, got {t.dtype}")
    return code


class Microscaled(NamedTuple):
    """Rows of `cols` values in a microscaled format (MX_FORMATS), padded to a
    multiple of 32: E4M3 codes with an E8M0 scale per 32 ("mxfp8"), E2M1 codes
    with an E8M0 scale per 32 ("mxfp4"), or E2M1 codes with an E4M3 scale per 16
    and a float32 scale per row ("nvfp4").  The layouts are those of
    include/fqa.h; allocate with alloc_microscaled()."""
    codes: torch.Tensor                  # uint8 [M, Kp], or [M, Kp / 2] for the 4-bit formats
    scales: torch.Tensor                 # uint8 [ceil(M/128), words, 32, 4, 4]
    row_scale: Optional[torch.Tensor]    # float32 [M], nvfp4 only
    cols: int
    fmt: str


def _mx_format(fmt) -> int:
    code = MX_FORMATS.get(fmt) if isinstance(fmt, str) else None
    if code is None:
        raise ValueError(f"fmt: expected one of {', '.join(MX_FORMATS)}, got {fmt!r}")
    return code


@functools.lru_cache(maxsize=1024, typed=True)
def _mx_shapes(M: int, K: int, code: int):
    """Shapes of the codes and of the scale tiles of [M, K]."""
    try:
        M, K = operator.index(M), operator.index(K)
    except TypeError:
        raise ValueError(f"[{M!r}, {K!r}]: expected whole numbers of rows and values") from None
    if not 0 <= M <= _MX_MAX_ROWS or not 1 <= K <= _MX_MAX_COLS:
        raise ValueError(f"[{M}, {K}]: microscaled rows are at most 2^24, of 1 to 2^20 values")
    kp = (K + 31) // 32 * 32
    width = 64 if code == 2 else 128
    return (M, kp if code == 0 else kp // 2), ((M + 127) // 128, (kp + width - 1) // width, 32, 4, 4)


def alloc_microscaled(M: int, K: int, fmt: str, device) -> Microscaled:
    code = _mx_format(fmt)
    codes, scales = _mx_shapes(M, K, code)
    return Microscaled(torch.empty(codes, dtype=torch.uint8, device=device),
                       torch.empty(scales, dtype=torch.uint8, device=device),
                       torch.empty(M, dtype=torch.float32, device=device) if code == 2 else None, operator.index(K), fmt)


def _require_microscaled(q, name: str, index: int = -1):
    """(rows, format code, device index) of a checked Microscaled."""
    if not isinstance(q, Microscaled):
        raise TypeError(f"{name}: expected a Microscaled, got {type(q).__name__}")
    codes, scales, row_scale, cols, fmt = q
    code = _mx_format(fmt)
    index = _device_tensor(codes, name + ".codes", index)
    if codes.dim() != 2:
        raise ValueError(f"{name}.codes: expected a 2-D tensor")
    M = codes.shape[0]
    code_shape, scale_shape = _mx_shapes(M, cols, code)
    _device_tensor(scales, name + ".scales", index)
    if code == 2:
        _device_tensor(row_scale, name + ".row_scale", index)
        if row_scale.dtype != torch.float32 or row_scale.shape != (M,) or not row_scale.is_contiguous():
            raise ValueError(f"{name}.row_scale: expected contiguous float32 [{M}], "
                             f"got {row_scale.dtype} {tuple(row_scale.shape)}")
    elif row_scale is not None:
        raise ValueError(f"{name}.row_scale: {fmt} rows have none")
    for t, part, shape in ((codes, "codes", code_shape), (scales, "scales", scale_shape)):
        if t.dtype != torch.uint8 or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}.{part}: expected a contiguous uint8 tensor of shape {shape}, "
                             f"got {t.dtype} {tuple(t.shape)}")
    return M, code, index


def _rows(x, name: str):
    """(rows, row length, row stride) of a tensor [..., K] with adjacent channels."""
    if x.dim() < 2:
        raise ValueError(f"{name}: expected [..., K] with at least two dimensions, got {tuple(x.shape)}")
    if x.dim() > 2:
        try:
            x = x.view(-1, x.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}: the leading dimensions have no common row stride") from None
    M, K = x.shape
    if K > 1 and x.stride(1) != 1:
        raise ValueError(f"{name}: expected adjacent channels, got stride {x.stride(1)}")
    return M, K, x.stride(0) if M > 1 else K


def _require_mx_out(out, fmt: str, M: int, K: int, code: int, index: int, inputs) -> None:
    if _require_microscaled(out, "out", index)[:2] != (M, code) or out.cols != K:
        raise ValueError(f"out: expected {fmt} rows [{M}, {K}]")
    parts = [t for t in out[:3] if t is not None]
    for i, t in enumerate(parts):
        _apart(t, "out", (*inputs, *parts[:i]))


def mx_quantize(x: torch.Tensor, fmt: str, out: Optional[Microscaled] = None, stream=None) -> Microscaled:
    """Rows [..., K] of bfloat16, float16 or float32 -> Microscaled rows (leading
    dimensions flattened).  A block (nvfp4: a row) with a NaN or an infinity
    stands for NaN."""
    if out is None and stream is None and (q := (_native or _native_calls()).quantize(x, fmt)) is not None:
        return q
    index = _device_tensor(x, "x")
    if (there := _elsewhere(index, stream, (x, *(() if out is None else out[:3])))) is not None:
        with there:
            return mx_quantize(x, fmt, out)
    dtype, code = _float_dtype(x, "x"), _mx_format(fmt)
    M, K, ld = _rows(x, "x")
    if out is None:
        out = alloc_microscaled(M, K, fmt, x.device)
    else:
        _require_mx_out(out, fmt, M, K, code, index, (x,))
    _check(_load().fqa_mx_quantize(x.data_ptr(), dtype, M, K, ld, code, out.codes.data_ptr(), out.scales.data_ptr(),
                                   _at(out.row_scale), _raw_stream(index)), "fqa_mx_quantize")
    return out


def mx_dequantize(q: Microscaled, out_dtype: int = FQA_OUT_BF16, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """The values that microscaled rows stand for, [M, cols]."""
    if out is None and stream is None and (v := (_native or _native_calls()).dequantize(q, out_dtype)) is not None:
        return v
    M, code, index = _require_microscaled(q, "q")
    if (there := _elsewhere(index, stream, (*q[:3], out))) is not None:
        with there:
            return mx_dequantize(q, out_dtype, out)
    dt = _OUT_DTYPE.get(out_dtype)
    if dt is None:
        raise ValueError(f"out_dtype: unknown value {out_dtype!r}")
    if out is None:
        out = torch.empty((M, q.cols), dtype=dt, device=q.codes.device)
    else:
        _device_tensor(out, "out", index)
        _require(out, dt, "out", (M, q.cols))
        _apart(out, "out", q[:3])
    _check(_load().fqa_mx_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), _at(q.row_scale), M, q.cols, code,
                                     out.data_ptr(), out_dtype, _raw_stream(index)), "fqa_mx_dequantize")
    return out


def mx_rms_norm(x: torch.Tensor, weight: torch.Tensor, fmt: str = "mxfp8", residual: Optional[torch.Tensor] = None,
                eps: float = 1e-6, out: Optional[Microscaled] = None, residual_out: Optional[torch.Tensor] = None,
                stream=None):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight over the rows of
    [..., K]: (y as Microscaled rows, h in residual's type, or None without a
    residual).  weight [K] and residual are of x's type or float32.
    residual_out may be residual itself (or x, where of the same type)."""
    if out is None and residual_out is None and stream is None and (
            y := (_native or _native_calls()).rms_norm(x, weight, fmt, residual, eps)) is not None:
        return y
    index = _device_tensor(x, "x")
    if (there := _elsewhere(index, stream, (x, weight, residual, residual_out, *(() if out is None else out[:3])))) is not None:
        with there:
            return mx_rms_norm(x, weight, fmt, residual, eps, out, residual_out)
    dtype, code = _float_dtype(x, "x"), _mx_format(fmt)
    M, K, ld = _rows(x, "x")
    _device_tensor(weight, "weight", index)
    if weight.shape != (K,) or weight.dtype not in (x.dtype, torch.float32) or not weight.is_contiguous():
        raise ValueError(f"weight: expected contiguous [{K}] of {x.dtype} or float32, "
                         f"got {tuple(weight.shape)} {weight.dtype}")
    if not 0.0 <= eps < float("inf"):
        raise ValueError(f"eps: expected a finite value of at least 0, got {eps}")
    ldr, res_dtype = K, dtype
    if residual is not None:
        _device_tensor(residual, "residual", index)
        if residual.shape != x.shape or residual.dtype not in (x.dtype, torch.float32):
            raise ValueError(f"residual: expected {tuple(x.shape)} of {x.dtype} or float32, "
                             f"got {tuple(residual.shape)} {residual.dtype}")
        ldr, res_dtype = _rows(residual, "residual")[2], _DTYPE[residual.dtype]
        if residual_out is None:
            residual_out = torch.empty(x.shape, dtype=residual.dtype, device=x.device)
        else:
            _device_tensor(residual_out, "residual_out", index)
            _require(residual_out, residual.dtype, "residual_out", x.shape)
            _apart(residual_out, "residual_out",
                   [weight] + [t for t in (x, residual) if not _same_memory(residual_out, t)])
    elif residual_out is not None:
        raise ValueError("residual_out: there is no residual")
    if out is None:
        out = alloc_microscaled(M, K, fmt, x.device)
    else:
        _require_mx_out(out, fmt, M, K, code, index, (x, weight, residual, residual_out))
    _check(_load().fqa_mx_rms_norm(
        x.data_ptr(), dtype, M, K, ld, weight.data_ptr(), _DTYPE[weight.dtype], eps, _at(residual), res_dtype, ldr, code,
        out.codes.data_ptr(), out.scales.data_ptr(), _at(out.row_scale), _at(residual_out), _raw_stream(index)),
        "fqa_mx_rms_norm")
    return out, residual_out


def mx_matmul(a: Microscaled, b: Microscaled, bias: Optional[torch.Tensor] = None, out_dtype: int = FQA_OUT_BF16,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """a [M, K] times the transpose of b [N, K] (a projection's weights), both
    microscaled rows of one format, plus a float32 bias [N]: [M, N]."""
    if out is None and stream is None and (y := (_native or _native_calls()).matmul(a, b, bias, out_dtype)) is not None:
        return y
    M, code, index = _require_microscaled(a, "a")
    N, other, _ = _require_microscaled(b, "b", index)
    if (there := _elsewhere(index, stream, (*a[:3], *b[:3], bias, out))) is not None:
        with there:
            return mx_matmul(a, b, bias, out_dtype, out)
    if other != code or a.cols != b.cols:
        raise ValueError(f"a and b: {a.fmt} rows of {a.cols} against {b.fmt} rows of {b.cols}")
    dt = _OUT_DTYPE.get(out_dtype)
    if dt is None:
        raise ValueError(f"out_dtype: unknown value {out_dtype!r}")
    if bias is not None:
        _device_tensor(bias, "bias", index)
        _require(bias, torch.float32, "bias", (N,))
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=a.codes.device)
    else:
        _device_tensor(out, "out", index)
        _require(out, dt, "out", (M, N))
        _apart(out, "out", (*a[:3], *b[:3], bias))
    _check(_load().fqa_mx_matmul(a.codes.data_ptr(), a.scales.data_ptr(), _at(a.row_scale), b.codes.data_ptr(),
                                 b.scales.data_ptr(), _at(b.row_scale), _at(bias), M, N, a.cols, code, out.data_ptr(),
                                 out_dtype, _raw_stream(index)), "fqa_mx_matmul")
    return out


class Rotary(NamedTuple):
    """Rotary positions for rotary() and the attention paths: positions int32 or
    float32 [N, A] or [B, N, A] for A axes (1..4), axes the channels of each
    (even, together at most 128; the rest is not rotated).  `split` pairs
    channels (j, D/2 + j) instead of (2j, 2j + 1), D = sum(axes), then a multiple
    of 16; `shared` takes one spectrum theta^(-2j/D) over all axes instead of
    theta^(-2i/axes[a]) on each.  q_weight and k_weight [128] (of q's type): RMS
    norm of each head before the rotation."""
    positions: torch.Tensor
    axes: tuple
    theta: float = 10000.0
    split: bool = False
    shared: bool = False
    q_weight: Optional[torch.Tensor] = None
    k_weight: Optional[torch.Tensor] = None
    eps: float = 1e-6


def _axes_array(axes: tuple, split: bool):
    # (types here: the cache takes 64.0 for 64)
    if any(not isinstance(a, int) for a in axes):
        raise ValueError(f"axes: expected whole channel counts, got {axes}")
    return _axes_of(axes, split)


@functools.lru_cache(maxsize=64)
def _axes_of(axes: tuple, split: bool):
    if not 1 <= len(axes) <= 4 or any(a < 2 or a % 2 for a in axes) or sum(axes) > HEAD_DIM:
        raise ValueError(f"axes: expected one to four even channel counts, together at most {HEAD_DIM}, got {axes}")
    if split and sum(axes) % 16:
        raise ValueError(f"axes: split pairs need a multiple of 16 channels, got {sum(axes)}")
    return (ctypes.c_int * len(axes))(*axes)


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], rot: Rotary, inverse: bool = False,
           q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Q [B,Hq,N,128] and K [B,Hk,N,128] (any strides over batch, heads and tokens,
    adjacent channels; k may be None) -> both normalized (where rot has
    weights) and rotated, contiguous.  `inverse` rotates back.  An output may be
    its own input where that is contiguous."""
    if q_out is None and k_out is None and stream is None and (
            y := (_native or _native_calls()).rotate(q, k, rot, inverse)) is not None:
        return y
    index = _device_tensor(q, "q")
    if not isinstance(rot, Rotary):
        raise TypeError(f"rot: expected a Rotary, got {type(rot).__name__}")
    pos, axes, theta, split, shared, q_weight, k_weight, eps = rot
    if (there := _elsewhere(index, stream, (q, k, pos, q_weight, k_weight, q_out, k_out))) is not None:
        with there:
            return rotary(q, k, rot, inverse, q_out, k_out)
    dtype = _float_dtype(q, "q")
    if q.dim() != 4:
        raise ValueError("q: expected a [B, H, N, 128] tensor")
    B, Hq, N, d = q.shape
    if d != HEAD_DIM:
        raise ValueError(f"q: expected {HEAD_DIM} channels, got {d}")
    sb, sh, sn, sd = q.stride()
    kb = kh = kn = Hk = 0
    kd = 1
    if k is not None:
        _device_tensor(k, "k", index)
        if k.dim() != 4 or k.dtype != q.dtype or k.shape[0] != B or k.shape[2] != N or k.shape[3] != d:
            raise ValueError(f"k: expected [{B}, H, {N}, {d}] of {q.dtype}, got {tuple(k.shape)} {k.dtype}")
        Hk = k.shape[1]
        kb, kh, kn, kd = k.stride()
    elif k_out is not None:
        raise ValueError("k_out: there is no k")
    if sd != 1 or kd != 1:
        raise ValueError(f"q and k: expected adjacent channels, got strides {sd} and {kd}")
    array, A = _axes_array(axes if isinstance(axes, tuple) else tuple(axes), bool(split)), len(axes)
    _device_tensor(pos, "rot.positions", index)
    shape = pos.shape
    if pos.dtype not in (torch.int32, torch.float32) or not pos.is_contiguous() or (
            shape != (N, A) and shape != (B, N, A) and shape != (1, N, A)):
        raise ValueError(f"rot.positions: expected contiguous int32 or float32 [{N}, {A}] or [{B}, {N}, {A}], "
                         f"got {pos.dtype} {tuple(shape)}")
    for name, w in (("rot.q_weight", q_weight), ("rot.k_weight", k_weight)):
        if w is not None:
            _device_tensor(w, name, index)
            if w.dtype != q.dtype or w.shape != (HEAD_DIM,) or not w.is_contiguous():
                raise ValueError(f"{name}: expected contiguous [{HEAD_DIM}] of {q.dtype}, got {w.dtype} {tuple(w.shape)}")
    if not 0.0 < theta < float("inf") or not 0.0 <= eps < float("inf"):
        raise ValueError(f"rot: expected a finite theta > 0 and eps >= 0, got {theta} and {eps}")
    if q_out is None and k_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        weights = (pos, q_weight, k_weight)
        for name, o, own, others in (("q_out", q_out, q, (k, *weights)), ("k_out", k_out, k, (q, *weights))):
            if o is not None:
                _device_tensor(o, name, index)
                _require(o, q.dtype, name, own.shape)
                _apart(o, name, others if _same_memory(o, own) else (own, *others))
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif k_out is not None:
            _apart(k_out, "k_out", (q_out,))
    if k is not None and k_out is None:
        k_out = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    _check(_load().fqa_rotary(
        q.data_ptr(), _at(k), dtype, B, Hq, Hk, N, d, sb, sh, sn, kb, kh, kn, pos.data_ptr(), _DTYPE[pos.dtype],
        N * A if len(shape) == 3 and shape[0] > 1 else 0, A, array, theta,
        (1 if split else 0) | (2 if shared else 0) | (4 if inverse else 0), _at(q_weight), _at(k_weight), eps,
        q_out.data_ptr(), _at(k_out), _raw_stream(index)), "fqa_rotary")
    return q_out, k_out


def softmax_scale(d: int = HEAD_DIM) -> float:
    """fl32(1/sqrt(d))."""
    return float(torch.tensor(1.0, dtype=torch.float32) / torch.sqrt(torch.tensor(float(d), dtype=torch.float32)))
