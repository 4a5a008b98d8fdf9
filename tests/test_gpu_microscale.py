"""Microscaled quantization, the RMS norm into it and the way back, on the GPU
against the 64-bit reference."""

import numpy as np
import pytest
import torch

from tests import block_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def fqa():
    import quantized_fp8_attention_b200 as f
    return f


def rand(M, K, dt, seed, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, device="cuda", generator=g)
    return (x * torch.exp(spread * torch.randn(M, 1, device="cuda", generator=g))).to(DT[dt])


def same_as_reference(q, x64):
    codes, bytes_, row = R.held(q)
    rc, rb, rr = R.quantize(x64, q.fmt)
    assert np.array_equal(bytes_, rb)
    if rr is not None:
        assert np.array_equal(row, rr, equal_nan=True)
    # a block or row that stands for NaN holds zero codes whatever their sign
    dead = np.repeat(rb == 255, R.BLOCK[q.fmt], 1) if rr is None else np.isnan(rr)[:, None] & np.ones_like(rc, bool)
    assert np.array_equal(np.where(dead, 0, codes), np.where(dead, 0, rc))
    assert not codes[dead].any()


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("M,K,dt", [
    (1, 1, "bf16"), (1, 32, "f32"), (3, 33, "f16"), (5, 100, "bf16"), (129, 64, "f16"), (7, 1000, "f32"),
    (2, 1024, "bf16"), (2, 1025, "bf16"), (130, 2001, "f16"), (4, 4096, "f32"), (3, 5100, "bf16"),
    (2, 16384, "bf16"), (3, 16392, "f16"), (2, 20001, "bf16"), (1, 70000, "f32")])
def test_quantize_is_exact(fmt, M, K, dt):
    x = rand(M, K, dt, M + K)
    same_as_reference(fqa().mx_quantize(x, fmt), x.double().cpu().numpy())


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_special_rows(fmt):
    """Zeros, ties of every code, tiny and huge magnitudes, infinities and NaN."""
    x = torch.zeros(12, 96, device="cuda")
    x[1, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4, device="cuda")
    x[2] = x[1] * -15.0                      # ties under a scale whose reciprocal rounds up
    x[3, 7] = 1e-45
    x[4] = 1e-38
    x[5, 50] = 3e38
    x[6, 33] = float("inf")
    x[7, 95] = float("nan")
    x[8, 0], x[8, 40] = -float("inf"), float("nan")
    x[9] = -0.0
    x[10] = torch.linspace(-448, 448, 96, device="cuda")
    x[11, ::16] = 2688.0 * 2.0 ** -130
    same_as_reference(fqa().mx_quantize(x, fmt), x.double().cpu().numpy())


def test_nvfp4_ties_under_every_scale():
    """x = s * t for every E4M3 scale s and every midpoint t of E2M1: the code is
    the even neighbour's, as in exact arithmetic."""
    s = torch.from_numpy(R.E4M3[1:]).float()
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = torch.zeros(126, 32)
    x[:, 0] = 6 * s
    x[:, 1:8] = s[:, None] * mids
    x[:, 8:15] = -x[:, 1:8]
    x[:, 16] = 2688.0                        # pins the row scale to 1
    same_as_reference(fqa().mx_quantize(x.cuda(), "nvfp4"), x.double().numpy())


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_strided_rows_and_leading_dimensions(fmt):
    f = fqa()
    wide = rand(37, 300, "bf16", 1)
    for x in (wide[:, 8:264], wide[:, 3:259], wide[::2, :96], wide[:1].expand(5, 300)):
        same_as_reference(f.mx_quantize(x, fmt), x.double().cpu().numpy())
    x = rand(24, 64, "bf16", 2).view(2, 3, 4, 64)
    same_as_reference(f.mx_quantize(x, fmt), x.double().cpu().numpy().reshape(24, 64))
    x = rand(64, 24, "f32", 2).T[:, :1]      # one channel
    same_as_reference(f.mx_quantize(x, fmt), x.double().cpu().numpy())


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_rows_past_the_end_are_left_alone(fmt):
    f = fqa()
    M, K = 133, 160
    out = f.alloc_microscaled(M, K, fmt, "cuda")
    big = torch.full((out.codes.numel() + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    out.scales.fill_(0x5A)
    out = out._replace(codes=big[: out.codes.numel()].view(out.codes.shape))
    x = rand(M, K, "bf16", 5)
    f.mx_quantize(x, fmt, out=out)
    same_as_reference(out, x.double().cpu().numpy())
    assert (big[out.codes.numel():] == 0x5A).all()
    words = out.scales.cpu().numpy()
    r, j = np.arange(M, 256)[:, None], np.arange(4 * words.shape[1])[None]
    assert (words[r // 128, j // 4, r % 32, r // 32 % 4, j % 4] == 0x5A).all()
    # blocks past Kp of a row's last word are written as 0
    blocks = K // R.BLOCK[fmt]
    r = np.arange(M)[:, None]
    j = np.arange(blocks, 4 * words.shape[1])[None]
    assert (words[r // 128, j // 4, r % 32, r // 32 % 4, j % 4] == 0).all()


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("out_dtype", [0, 1, 2])
@pytest.mark.parametrize("M,K", [(1, 1), (130, 77), (5, 4096), (257, 320)])
def test_dequantize(fmt, out_dtype, M, K):
    f = fqa()
    q = R.random_microscaled(M, K, fmt, M + K, wide=True)
    got = f.mx_dequantize(q, out_dtype)
    assert got.dtype == f._OUT_DTYPE[out_dtype] and got.shape == (M, K)
    want = R.values(*R.held(q), fmt, K)
    # code * scale is exact in binary32; the row scale's product rounds once
    # there and the output once more
    half = torch.finfo(got.dtype).eps / 2 + (2.0 ** -24 if fmt == "nvfp4" else 0.0)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= half * 1.001 * np.abs(want) + (2.0 ** -25 if out_dtype == 2 else 0.0)).all()


def test_dequantize_gives_nan_for_nan_blocks():
    f = fqa()
    x = torch.ones(3, 96, device="cuda")
    x[1, 40] = float("inf")
    for fmt in R.FORMATS:
        v = f.mx_dequantize(f.mx_quantize(x, fmt))
        bad = torch.isnan(v)
        assert bad[1, 32:64].all() and not bad[0].any() and not bad[2].any()
        assert bad[1].all() == (fmt == "nvfp4")


# ------------------------------------------------------------------ norm

def check_norm(x, weight, residual, fmt, eps, q, h, d=2.0 ** -18):
    """y carries at most 64 binary32 roundings (the sum of squares: at most 40 in
    a thread and 14 across threads, halved by the root; division, eps, rsqrtf
    two units, two products, the sum h): |dy| <= 2^-18 |y|.  The codes have to
    be the rounding of some value that near, under the scale the row got."""
    K = x.shape[-1]
    y, h64 = R.rms_norm(x.reshape(-1, K), weight, None if residual is None else residual.reshape(-1, K), eps)
    if residual is not None:
        got = h.reshape(-1, K).double().cpu().numpy()
        assert h.dtype == residual.dtype
        # binary32 sum, then one rounding to the residual's type
        half = torch.finfo(h.dtype).eps / 2 + (2.0 ** -24 if h.dtype != torch.float32 else 0.0)
        tiny = 2.0 ** -25 if h.dtype == torch.float16 else 0.0
        assert (np.abs(got - h64) <= 1.001 * half * np.abs(h64) + tiny).all()
    else:
        assert h is None
    codes, bytes_, row = R.held(q)
    lo_scale, hi_scale = R.quantize(y * (1 - d), fmt), R.quantize(y * (1 + d), fmt)
    assert ((bytes_ >= np.minimum(lo_scale[1], hi_scale[1])) & (bytes_ <= np.maximum(lo_scale[1], hi_scale[1]))).all() \
        or fmt == "nvfp4"
    if row is not None:
        assert ((row >= lo_scale[2]) & (row <= hi_scale[2])).all()
    # what one unit of the code's grid spans, under the scales that were written
    table = R.E4M3 if fmt == "mxfp8" else R.E2M1
    M = y.shape[0]
    full = np.zeros((M, codes.shape[1]))
    full[:, :K] = y
    scale = R.E4M3[bytes_ & 127] if fmt == "nvfp4" else 2.0 ** (bytes_.astype(int) - 127.0)
    step = np.repeat(scale, R.BLOCK[fmt], 1) * (1.0 if row is None else row[:, None])
    safe = np.where(step > 0, step, 1.0)
    a, b = (R.nearest(np.abs(full) * f / safe, table) for f in (1 - d, 1 + d))
    mag = codes & (127 if fmt == "mxfp8" else 7)
    assert (((mag >= a) & (mag <= b)) | (step == 0)).all()
    assert not codes[step == 0].any()
    if fmt == "nvfp4":
        # each block's scale: the E4M3 rounding of amax / 6 row, within d
        amax = np.abs(full).reshape(M, -1, 16).max(2) / row[:, None] / 6
        assert ((bytes_ >= R.nearest(amax * (1 - d), R.E4M3)) & (bytes_ <= R.nearest(amax * (1 + d), R.E4M3))).all()
    sign = (codes & (128 if fmt == "mxfp8" else 8)) != 0
    assert (sign == np.signbit(full))[mag > 0].all()


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("M,K,dt,res,wt", [
    (1, 1, "bf16", None, "bf16"), (1, 4096, "bf16", "bf16", "bf16"), (5, 96, "f32", "f32", "f32"),
    (3, 1000, "f16", "f32", "f16"), (130, 1024, "bf16", "f32", "f32"), (4, 1031, "bf16", "bf16", "f32"),
    (9, 5100, "f32", "f32", "f32"), (2, 16384, "f16", "f16", "f16"), (3, 16416, "bf16", "bf16", "bf16"),
    (2, 20001, "f32", None, "f32")])
def test_norm(fmt, M, K, dt, res, wt):
    f = fqa()
    x = rand(M, K, dt, K, 1.0)
    weight = (1 + 0.3 * torch.randn(K, device="cuda")).to(DT[wt])
    residual = None if res is None else rand(M, K, res, K + 1, 1.0)
    q, h = f.mx_rms_norm(x, weight, fmt, residual=residual, eps=1e-5)
    check_norm(x, weight, residual, fmt, 1e-5, q, h)


@pytest.mark.parametrize("K", [512, 2048, 8192, 20000])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_norm_in_place_equals_out_of_place(K, fmt):
    """residual_out = residual, and = x: every path, the one that reads a long row
    again too."""
    f = fqa()
    x, r = rand(6, K, "bf16", 1, 1.0), rand(6, K, "bf16", 2, 1.0)
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    q, h = f.mx_rms_norm(x, w, fmt, residual=r)
    for which in (0, 1):
        xc, rc = x.clone(), r.clone()
        q2, h2 = f.mx_rms_norm(xc, w, fmt, residual=rc, residual_out=(rc, xc)[which])
        assert h2.data_ptr() == (rc, xc)[which].data_ptr() and torch.equal(h, h2)
        for a, b in zip(R.held(q), R.held(q2)):
            assert (a is None and b is None) or np.array_equal(a, b)


def test_norm_of_strided_and_broadcast_rows():
    f = fqa()
    wide = rand(40, 520, "bf16", 3, 1.0)
    w = (1 + 0.1 * torch.randn(256, device="cuda")).bfloat16()
    for x, r in ((wide[:, 8:264], wide[:, 264:520]), (wide[:, 1:257], wide[:, 257:513]),
                 (wide[:, :256], wide[:1, :256].expand(40, 256))):
        q, h = f.mx_rms_norm(x, w, "mxfp8", residual=r)
        check_norm(x, w, r, "mxfp8", 1e-6, q, h)
        assert h.is_contiguous()
    x3 = rand(24, 64, "f32", 4, 1.0).view(2, 3, 4, 64)
    q, h = f.mx_rms_norm(x3, torch.ones(64, device="cuda"), "nvfp4", residual=x3)
    assert h.shape == x3.shape and torch.equal(h, x3 + x3)


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_norm_of_zero_and_non_finite_rows(fmt):
    """A zero row (eps > 0) gives zeros; eps = 0 makes it 0 * inf = NaN; an
    infinity makes its own element NaN and the rest 0; NaN spoils its row.  Other
    rows keep their values."""
    f = fqa()
    x = rand(6, 160, "f32", 7, 0.0)
    x[1] = 0
    x[2, 50] = float("inf")
    x[3, 3] = float("nan")
    w = torch.ones(160, device="cuda")
    clean = rand(6, 160, "f32", 7, 0.0)
    v = f.mx_dequantize(f.mx_rms_norm(x, w, fmt)[0], 1)
    ref = f.mx_dequantize(f.mx_rms_norm(clean, w, fmt)[0], 1)
    for r in (0, 4, 5):
        assert torch.equal(v[r], ref[r])
    assert (v[1] == 0).all() and torch.isnan(v[3]).all()
    assert torch.isnan(v[2, 32:64]).all()
    assert torch.isnan(v[2]).all() if fmt == "nvfp4" else (v[2, :32] == 0).all() and (v[2, 64:] == 0).all()
    assert torch.isnan(f.mx_dequantize(f.mx_rms_norm(x, w, fmt, eps=0.0)[0], 1)[1]).all()


def test_empty_rows():
    f = fqa()
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for fmt in R.FORMATS:
        q = f.mx_quantize(x, fmt)
        assert q.codes.shape[0] == 0 and q.scales.numel() == 0 and f.mx_dequantize(q).shape == (0, 64)
        q, h = f.mx_rms_norm(x, w, fmt, residual=x)
        assert q.codes.shape[0] == 0 and h.shape == (0, 64)


def test_another_stream_and_a_replayed_graph():
    f = fqa()
    x, r = rand(64, 512, "bf16", 1, 1.0), rand(64, 512, "bf16", 2, 1.0)
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    want, hw = f.mx_rms_norm(x, w, "nvfp4", residual=r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, hg = f.mx_rms_norm(x, w, "nvfp4", residual=r, stream=side)
    side.synchronize()
    assert torch.equal(hw, hg) and all(np.array_equal(a, b) for a, b in zip(R.held(want), R.held(got)))
    xs, rs = torch.zeros_like(x), torch.zeros_like(r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, h = f.mx_rms_norm(xs, w, "nvfp4", residual=rs)
        v = f.mx_dequantize(q)
    xs.copy_(x)
    rs.copy_(r)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, hw) and torch.equal(v, f.mx_dequantize(want))


def test_refusals():
    f = fqa()
    x = torch.zeros(4, 64, device="cuda").bfloat16()
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    q = f.mx_quantize(x, "nvfp4")
    m = f.mx_quantize(x, "mxfp4")
    h = torch.zeros_like(x)
    for bad in (lambda: f.mx_quantize(x, "mxfp6"), lambda: f.mx_quantize(x, 0), lambda: f.mx_quantize(x[0], "mxfp8"),
                lambda: f.mx_quantize(x.T, "mxfp8"), lambda: f.mx_quantize(x.int(), "mxfp8"),
                lambda: f.mx_quantize(x[:, :0], "mxfp8"), lambda: f.mx_quantize(x, "mxfp4", out=q),
                lambda: f.mx_quantize(x, "mxfp4", out=h), lambda: f.mx_rms_norm(x, w, out=h),
                lambda: f.mx_quantize(x[:3], "nvfp4", out=q), lambda: f.mx_quantize(x[:, :32], "nvfp4", out=q),
                lambda: f.mx_quantize(x, "mxfp4", out=m._replace(codes=x.view(torch.uint8)[:, :32])),
                lambda: f.mx_quantize(x, "mxfp4", out=m._replace(codes=x.view(torch.uint8).flatten()[:128].view(4, 32))),
                lambda: f.mx_dequantize(q._replace(row_scale=None)), lambda: f.mx_dequantize(m._replace(row_scale=q.row_scale)),
                lambda: f.mx_dequantize(q._replace(cols=65)), lambda: f.mx_dequantize(q, 3),
                lambda: f.mx_dequantize(q._replace(scales=q.scales[..., :2])), lambda: f.mx_dequantize(q, out=x[:3]),
                lambda: f.mx_rms_norm(x, w[:32]), lambda: f.mx_rms_norm(x, w.half()), lambda: f.mx_rms_norm(x, w, eps=-1.0),
                lambda: f.mx_rms_norm(x, w, residual=x[:2]), lambda: f.mx_rms_norm(x, w, residual=x.half()),
                lambda: f.mx_rms_norm(x, w, residual_out=h), lambda: f.mx_rms_norm(x, w, residual=x, residual_out=h.float()),
                lambda: f.mx_rms_norm(x[1:], w, residual=x[:3], residual_out=x[:3]),
                lambda: f.mx_matmul(q, m), lambda: f.mx_matmul(q, f.mx_quantize(x[:, :32], "nvfp4")),
                lambda: f.mx_matmul(q, q, bias=w[:4]), lambda: f.mx_matmul(q, q, out_dtype=7),
                lambda: f.mx_matmul(q, q, out=h[:, :4]), lambda: f.mx_matmul(q, q, bias=torch.zeros(5, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            bad()


def test_the_short_way_and_the_checked_one_agree():
    """The native everyday calls are the ones that run, and give what the Python
    functions give where an output or a stream sends them the other way."""
    f = fqa()
    f.lib()
    b = f._native
    x, r = rand(33, 200, "bf16", 1, 1.0), rand(33, 200, "f32", 2, 1.0)
    w = (1 + 0.1 * torch.randn(200, device="cuda")).bfloat16()
    bias = torch.randn(33, device="cuda")
    same = lambda p, q: all((s is None and t is None) or (torch.equal(s, t) if isinstance(s, torch.Tensor) else s == t)
                            for s, t in zip(p._replace(scales=None), q._replace(scales=None))) and all(
        np.array_equal(s, t) for s, t in zip(R.held(p)[:2], R.held(q)[:2]))
    here = torch.cuda.current_stream()
    for fmt in R.FORMATS:
        q = b.quantize(x, fmt)
        assert same(q, f.mx_quantize(x, fmt, stream=here))
        y, h = b.rms_norm(x, w, fmt, r, 1e-5)
        y2, h2 = f.mx_rms_norm(x, w, fmt, residual=r, eps=1e-5, stream=here)
        assert same(y, y2) and torch.equal(h, h2)
        for t in (0, 1, 2):
            assert torch.equal(b.dequantize(q, t), f.mx_dequantize(q, t, stream=here))
            assert torch.equal(b.matmul(y, q, bias, t), f.mx_matmul(y, q, bias=bias, out_dtype=t, stream=here))
    packed = torch.randn(2, 30, 5, 128, device="cuda").half()
    q, k = packed[:, :, :3].transpose(1, 2), packed[:, :, 3:].transpose(1, 2)
    rot = f.Rotary(torch.randint(0, 99, (30, 2), dtype=torch.int32, device="cuda"), (64, 64), split=True,
                   q_weight=torch.ones(128, device="cuda").half())
    for got, want in zip(b.rotate(q, k, rot, True), f.rotary(q, k, rot, inverse=True, stream=here)):
        assert torch.equal(got, want)
    # not the everyday call
    assert b.quantize(x[0], "mxfp8") is None and b.quantize(x.T, "mxfp8") is None and b.quantize(x, "mxfp6") is None
    assert b.matmul(q, q, None, 0) is None and b.matmul(y, y, bias[:3], 0) is None
    assert b.rotate(q, k[:, :, :3], rot, False) is None and b.rotate(q, k, rot._replace(axes=[64, 64]), False) is None


# off the 16-byte boundaries: one value, two and four an access, lengths around a
# CTA's steps, the longest row that is held on chip (49152 with its padding) and
# the next
OFF = [15, 18, 255, 258, 2047, 2050, 4097, 4098, 4100, 49118, 49151, 49153, 49154, 60001]


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("K", OFF)
def test_rows_off_the_boundaries(fmt, dt, K):
    f = fqa()
    x = rand(3, K, dt, K)
    q = f.mx_quantize(x, fmt)
    same_as_reference(q, x.double().cpu().numpy())
    # the way back: exact in BF16 but for the row scales' binary32 product
    v = f.mx_dequantize(q, 0).double().cpu().numpy()
    want = R.values(*R.held(q), fmt, K)
    assert (np.abs(v - want) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(want)).all()
    # and a view that starts inside a 16-byte piece holds what its copy holds
    y = rand(3, K + 3, dt, K + 1)[:, 1:K + 1]
    for a, b in zip(R.held(f.mx_quantize(y, fmt)), R.held(f.mx_quantize(y.clone(), fmt))):
        assert (a is None and b is None) or np.array_equal(a, b)


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("dt,res,wt", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "f32", "f32"),
                                       ("f16", None, "f32")])
@pytest.mark.parametrize("K", OFF)
def test_norm_off_the_boundaries(fmt, dt, res, wt, K):
    f = fqa()
    x = rand(3, K, dt, K, 1.0)
    weight = (1 + 0.3 * torch.randn(K, device="cuda")).to(DT[wt])
    residual = None if res is None else rand(3, K, res, K + 1, 1.0)
    q, h = f.mx_rms_norm(x, weight, fmt, residual=residual, eps=1e-5)
    # a thread adds up to 49152 / 256 = 192 squares in a row: (192 + 14) / 2 + 10
    # roundings are 113 <= 2^7 of 2^-24
    check_norm(x, weight, residual, fmt, 1e-5, q, h, 2.0 ** -17)
    if res == dt:
        for which in (0, 1):                     # residual_out = residual, and = x
            xc, rc = x.clone(), residual.clone()
            q2, h2 = f.mx_rms_norm(xc, weight, fmt, residual=rc, residual_out=(rc, xc)[which], eps=1e-5)
            assert torch.equal(h, h2)
            for a, b in zip(R.held(q), R.held(q2)):
                assert (a is None and b is None) or np.array_equal(a, b)


@pytest.mark.parametrize("K", [4096, 4097])
def test_rows_beyond_two_to_the_31_elements(K):
    """The last rows of 2.2e9 elements hold what they hold alone (both row paths)."""
    f = fqa()
    M = 128 * 4200 + 5
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    x[:200].normal_()
    x[200:-200] = 0
    x[-200:].normal_()
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    q = f.mx_quantize(x, "nvfp4")
    tail = f.mx_quantize(x[-133:].contiguous(), "nvfp4")
    assert torch.equal(q.codes[-133:], tail.codes) and torch.equal(q.row_scale[-133:], tail.row_scale)
    # row M - 133 starts a block of 128 rows, so the tiles line up (rows past M are not written)
    last, want = R.untile(q.scales[-2:], 133, 4), R.untile(tail.scales, 133, 4)
    assert np.array_equal(last, want)
    v = f.mx_dequantize(q)
    assert torch.equal(v[-133:], f.mx_dequantize(tail))
    del v
    y, h = f.mx_rms_norm(x, w, "mxfp8", residual=x)
    y2, h2 = f.mx_rms_norm(x[-133:].contiguous(), w, "mxfp8", residual=x[-133:].contiguous())
    assert torch.equal(y.codes[-133:], y2.codes) and torch.equal(h[-133:], h2)
