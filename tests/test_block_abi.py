"""Refusals of the microscaled and rotary calls: the C ABI's argument checks on
the host (addresses that are never read), and the binding's helpers, without a
GPU."""

import ctypes

import pytest
import torch

import quantized_fp8_attention_b200 as fqa

P = ctypes.c_void_p
OK = P(0x10000)


def at(n):
    return P(0x10000 + n)


@pytest.fixture(scope="module")
def L():
    from quantized_fp8_attention_b200 import build
    build.build()
    return fqa.lib()


def test_byte_counts(L):
    assert L.fqa_mx_code_bytes(5, 33, 0) == 5 * 64 and L.fqa_mx_code_bytes(5, 33, 1) == 5 * 32
    assert L.fqa_mx_scale_bytes(1, 1, 0) == 512                  # one tile of 128 rows x 4 blocks
    assert L.fqa_mx_scale_bytes(129, 129, 0) == 2 * 2 * 512      # Kp = 160: two words of 128 channels
    assert L.fqa_mx_scale_bytes(129, 129, 2) == 2 * 3 * 512      # three of 64
    for bad in ((-1, 32, 0), (1, 0, 0), (1, 32, 3), ((1 << 24) + 1, 32, 0), (1, (1 << 20) + 1, 0)):
        assert L.fqa_mx_code_bytes(*bad) == 0 and L.fqa_mx_scale_bytes(*bad) == 0
    for fmt, code in fqa.MX_FORMATS.items():
        for M, K in ((1, 1), (77, 2001), (300, 4096)):
            codes, scales = fqa._mx_shapes(M, K, code)
            assert L.fqa_mx_code_bytes(M, K, code) == codes[0] * codes[1]
            n = 1
            for s in scales:
                n *= s
            assert L.fqa_mx_scale_bytes(M, K, code) == n


def test_quantize_validation(L):
    def call(**kw):
        return L.fqa_mx_quantize(kw.get("x", OK), kw.get("dt", 0), kw.get("M", 4), kw.get("K", 64), kw.get("ld", 64),
                                 kw.get("fmt", 0), kw.get("codes", OK), kw.get("scales", OK), kw.get("row", OK), None)
    for kw in (dict(x=None), dict(codes=None), dict(scales=None), dict(M=-1), dict(K=0), dict(dt=3), dict(dt=-1),
               dict(fmt=3), dict(ld=-1), dict(fmt=2, row=None)):
        assert call(**kw) == 1, kw
    assert call(M=(1 << 24) + 1) == 2 and call(K=(1 << 20) + 1) == 2
    for kw in (dict(x=at(1)), dict(dt=1, x=at(2)), dict(codes=at(8)), dict(scales=at(4)), dict(fmt=2, row=at(2))):
        assert call(**kw) == 3, kw
    assert call(M=0, x=None, codes=None) == 0                    # no rows: nothing to do


def test_norm_validation(L):
    def call(**kw):
        return L.fqa_mx_rms_norm(kw.get("x", OK), kw.get("dt", 0), kw.get("M", 4), kw.get("K", 64), kw.get("ld", 64),
                                 kw.get("w", OK), kw.get("wdt", 0), kw.get("eps", 1e-6), kw.get("r", OK),
                                 kw.get("rdt", 0), kw.get("ldr", 64), kw.get("fmt", 0), OK, OK, OK, kw.get("ro", OK),
                                 None)
    for kw in (dict(x=None), dict(w=None), dict(r=None), dict(ro=None), dict(wdt=2), dict(rdt=2), dict(rdt=3),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(ldr=-1), dict(fmt=-1)):
        assert call(**kw) == 1, kw
    for kw in (dict(w=at(1)), dict(wdt=1, w=at(2)), dict(r=at(1)), dict(rdt=1, ro=at(2))):
        assert call(**kw) == 3, kw
    assert call(M=0, w=None) == 0


def test_dequantize_validation(L):
    def call(**kw):
        return L.fqa_mx_dequantize(kw.get("codes", OK), kw.get("scales", OK), kw.get("row", OK), kw.get("M", 4),
                                   kw.get("K", 64), kw.get("fmt", 0), kw.get("out", OK), kw.get("dt", 0), None)
    for kw in (dict(codes=None), dict(scales=None), dict(out=None), dict(fmt=2, row=None), dict(dt=3), dict(K=0)):
        assert call(**kw) == 1, kw
    assert call(K=1 << 21) == 2 and call(codes=at(4)) == 3 and call(dt=1, out=at(2)) == 3
    assert call(M=0, out=None) == 0


def test_matmul_validation(L):
    names = ("ac", "as_", "ar", "bc", "bs", "br")

    def call(**kw):
        return L.fqa_mx_matmul(*[kw.get(n, OK) for n in names], kw.get("bias", None), kw.get("M", 4), kw.get("N", 8),
                               kw.get("K", 64), kw.get("fmt", 2), kw.get("out", OK), kw.get("dt", 0), None)
    for kw in (*[{n: None} for n in names], dict(out=None), dict(M=-1), dict(N=-1), dict(K=0), dict(fmt=3), dict(dt=3)):
        assert call(**kw) == 1, kw
    assert call(M=(1 << 24) + 1) == 2 and call(N=(1 << 24) + 1) == 2 and call(K=(1 << 20) + 1) == 2
    for kw in (dict(ac=at(8)), dict(bs=at(8)), dict(ar=at(2)), dict(bias=at(2)), dict(out=at(1)), dict(dt=1, out=at(2))):
        assert call(**kw) == 3, kw
    assert call(M=0, out=None) == 0 and call(N=0, bc=None) == 0


def test_rotary_validation(L):
    def call(axes=(16, 56, 56), **kw):
        arr = (ctypes.c_int * len(axes))(*axes) if axes else None
        return L.fqa_rotary(kw.get("q", OK), kw.get("k", OK), kw.get("dt", 0), kw.get("B", 1), kw.get("Hq", 2),
                            kw.get("Hk", 2), kw.get("N", 3), kw.get("d", 128), *([768, 384, 128] * 2),
                            kw.get("pos", OK), kw.get("pdt", 3), kw.get("psb", 0), kw.get("n", len(axes)), arr,
                            kw.get("theta", 1e4), kw.get("flags", 0), kw.get("qw", None), kw.get("kw", None),
                            kw.get("eps", 1e-6), kw.get("qo", OK), kw.get("ko", OK), None)
    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(dt=3), dict(pdt=0),
               dict(B=-1), dict(N=-1), dict(Hq=-1), dict(n=0), dict(theta=0.0), dict(theta=float("inf")),
               dict(theta=float("nan")), dict(eps=-1.0), dict(flags=8), dict(psb=-1), dict(axes=(15, 57, 56)),
               dict(axes=(0, 64, 64)), dict(axes=(64, 64, 2)), dict(axes=(130,)), dict(axes=(-2, 64))):
        assert call(**kw) == 1, kw
    for kw in (dict(d=64), dict(axes=(2, 2, 2, 2, 2)), dict(flags=1, axes=(2, 4)), dict(B=1 << 16, N=1 << 16),
               dict(Hq=65535)):
        assert call(**kw) == 2, kw
    for kw in (dict(q=at(1)), dict(dt=1, k=at(2)), dict(qo=at(8)), dict(ko=at(4)), dict(pos=at(2)), dict(qw=at(1))):
        assert call(**kw) == 3, kw
    assert call(N=0, q=None) == 0 and call(B=0) == 0 and call(Hq=0, Hk=0, q=None, k=None) == 0


def test_host_tensors_are_refused():
    x = torch.zeros(4, 64)
    q = fqa.Microscaled(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), None, 64,
                        "mxfp8")
    rot = fqa.Rotary(torch.zeros(1, 1), (128,))
    for call in (lambda: fqa.mx_quantize(x, "mxfp8"), lambda: fqa.mx_rms_norm(x, x[0]), lambda: fqa.mx_dequantize(q),
                 lambda: fqa.mx_matmul(q, q), lambda: fqa.rotary(x, None, rot)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        fqa.mx_dequantize((1, 2))
    with pytest.raises(ValueError, match="fmt"):
        fqa.alloc_microscaled(1, 1, "fp3", "cpu")


def test_rows_and_extents():
    x = torch.zeros(6, 40)
    assert fqa._rows(x, "x") == (6, 40, 40)
    assert fqa._rows(x[:, 4:36], "x") == (6, 32, 40)
    assert fqa._rows(x[:1, :7], "x") == (1, 7, 7)
    assert fqa._rows(x[:1].expand(9, 40), "x") == (9, 40, 0)
    assert fqa._rows(x.view(2, 3, 40), "x") == (6, 40, 40)
    assert fqa._rows(torch.zeros(0, 8), "x") == (0, 8, 8)
    for bad in (x[0], x.T, torch.zeros(3, 2, 5).transpose(0, 1)):
        with pytest.raises(ValueError):
            fqa._rows(bad, "x")
    a = torch.zeros(100)
    fqa._apart(a[:50], "out", (a[50:], None, a[:0]))
    with pytest.raises(ValueError, match="overlaps"):
        fqa._apart(a[:51], "out", (a[50:],))
    with pytest.raises(ValueError, match="overlaps"):
        fqa._apart(a[1::2], "out", (a[::2],))       # interleaved: ranges cross
    assert fqa._same_memory(a, a) and not fqa._same_memory(a[:50:2], a[:50:2])


def test_axes():
    assert list(fqa._axes_array((16, 56, 56), False)) == [16, 56, 56]
    for axes, split in (((), False), ((1,), False), ((64, 66), False), ((2,) * 5, False), ((2, 4), True), ((8.0,), False)):
        with pytest.raises(ValueError):
            fqa._axes_array(axes, split)


def test_the_short_way_leaves_what_it_does_not_take_to_the_checks(L):
    """csrc/binding.cpp answers None to anything but the everyday call (here: host
    tensors, wrong types, wrong counts), and raises nothing."""
    from quantized_fp8_attention_b200 import _binding as b
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = fqa.Microscaled(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), None, 64,
                        "mxfp8")
    rot = fqa.Rotary(torch.zeros(1, 1), (128,))
    assert b.quantize(x, "mxfp8") is None and b.quantize(x) is None and b.quantize(3, "mxfp8") is None
    assert b.quantize(x, 7) is None and b.quantize(None, None) is None
    assert b.dequantize(q, 0) is None and b.dequantize((1, 2), 0) is None and b.dequantize(q, "0") is None
    assert b.rms_norm(x, x[0], "mxfp8", None, 1e-6) is None and b.rms_norm(x, x[0], "mxfp8", None, 1) is None
    assert b.matmul(q, q, None, 0) is None and b.matmul(q, None, None, 1 << 70) is None
    assert b.rotate(x, None, rot, False) is None and b.rotate(x, None, (1, 2), False) is None
