"""Products of microscaled rows on the block-scaled tensor cores, against the
same codes multiplied out in 64 bits."""

import numpy as np
import pytest
import torch

from tests import block_ref as R

pytestmark = pytest.mark.gpu


def fqa():
    import quantized_fp8_attention_b200 as f
    return f


def reference(a, b, bias):
    """(exact product, sum of |products|) on the GPU in binary64."""
    va, vb = (torch.from_numpy(R.values(*R.held(x), x.fmt, x.cols)).cuda() for x in (a, b))
    y = va @ vb.T
    mag = va.abs() @ vb.abs().T
    if bias is not None:
        y, mag = y + bias.double(), mag + bias.double().abs()
    return y, mag


def bound(y, mag, K, dtype):
    """Products of codes and scales are exact; each step of 32 values adds into a
    binary32 sum of magnitude at most `mag`, off by at most one unit (2^-23)
    whether it rounds or truncates; at most 8 partial sums, two row scales and
    the bias add 12 half units.  Then one rounding to the type."""
    eps = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return (K / 32 + 12) * 2.0 ** -23 * mag + eps * 1.01 * y.abs() + tiny


def check(M, N, K, fmt, out_dtype=1, bias=False, seed=0):
    f = fqa()
    a, b = R.random_microscaled(M, K, fmt, seed + 1, wide=True), R.random_microscaled(N, K, fmt, seed + 2, wide=True)
    bv = torch.randn(N, device="cuda") if bias else None
    canary = torch.full((M * N + 64,), -77.0, dtype=f._OUT_DTYPE[out_dtype], device="cuda")
    out = f.mx_matmul(a, b, bias=bv, out_dtype=out_dtype, out=canary[: M * N].view(M, N))
    torch.cuda.synchronize()
    assert f.fqa_debug_status()[0] == f.FQA_OK
    assert (canary[M * N:] == -77.0).all()
    y, mag = reference(a, b, bv)
    err = (out.double() - y).abs()
    lim = bound(y, mag, K, out.dtype)
    if out_dtype == 2:
        # FP16's largest value is 65504 and the next step 65536: what is nearer to
        # that (from 65520 on) becomes infinity; a sum within its own bound of
        # 65520 may fall on either side
        sure = y.abs() >= 65520 + bound(y, mag, K, torch.float32)
        either = y.abs() >= 65520 - bound(y, mag, K, torch.float32)
        assert torch.isinf(out[sure]).all()
        err, lim = err[~either], lim[~either]
    assert (err <= lim).all(), (float((err / lim).max()), M, N, K, fmt)


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 130, 64), (3, 127, 96), (16, 256, 256), (17, 100, 160),
    (31, 129, 1000), (32, 512, 2048), (33, 64, 320), (64, 200, 544), (65, 333, 96), (77, 2111, 4128), (127, 129, 224),
    (128, 128, 256), (129, 257, 288), (200, 384, 8192), (1, 64, 20000)])
def test_few_rows(fmt, M, N, K):
    check(M, N, K, fmt, bias=M % 2 == 1, seed=M + N + K)


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("M,N,K", [
    (256, 256, 32), (257, 511, 96), (300, 1000, 480), (513, 768, 1024), (1024, 4096, 256), (1000, 2056, 4096),
    (2048, 2304, 544), (4608, 1536, 1120), (3001, 2049, 64), (700, 8200, 33), (19000, 16, 64), (19100, 8, 96),
    (19001, 1, 32), (20000, 40, 288), (2500, 2304, 20000), (4000, 1282, 4128)])
def test_many_rows(fmt, M, N, K):
    check(M, N, K, fmt, bias=N % 2 == 0, seed=M + N + K)


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("out_dtype", [0, 1, 2])
@pytest.mark.parametrize("M,N,K", [(5, 200, 320), (90, 333, 640), (600, 1200, 800), (1500, 1999, 416)])
def test_output_types(fmt, out_dtype, M, N, K):
    check(M, N, K, fmt, out_dtype, bias=True, seed=3)


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("M", [3, 70, 1100, 3000])
def test_single_products_land_where_they_belong(fmt, M):
    """A's row m is one value at channel (7 m) % K, so every result is that value
    times one code of B: exact, and any misplaced row, channel or scale shows.
    The value is one that the format holds exactly: 1, or nvfp4's 6 * 448 * 2^-11
    (1 / 6 is no E4M3 scale)."""
    f = fqa()
    K, N = 352, 1090
    x = torch.zeros(M, K, device="cuda")
    unit = 1.3125 if fmt == "nvfp4" else 1.0
    x[torch.arange(M), (7 * torch.arange(M)) % K] = unit
    a, b = f.mx_quantize(x, fmt), R.random_microscaled(N, K, fmt, 5)
    want = torch.from_numpy(R.values(*R.held(b), fmt, K)).cuda()[:, (7 * torch.arange(M)) % K].T
    assert torch.equal(f.mx_matmul(a, b, out_dtype=1).double(), unit * want)


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("M,N", [(5, 300), (1200, 1100), (2600, 1300)])
def test_rows_that_stand_for_nan(fmt, M, N):
    """NaN in A's row m or B's row n spoils that row or column of the result only."""
    f = fqa()
    x, w = torch.randn(M, 200, device="cuda"), torch.randn(N, 200, device="cuda")
    clean = f.mx_matmul(f.mx_quantize(x, fmt), f.mx_quantize(w, fmt), out_dtype=1)
    x[3, 150], w[77, 10] = float("nan"), float("inf")
    y = f.mx_matmul(f.mx_quantize(x, fmt), f.mx_quantize(w, fmt), out_dtype=1)
    bad = torch.isnan(y)
    assert bad[3].all() and bad[:, 77].all()
    bad[3], bad[:, 77] = True, True
    assert not torch.isnan(y[~bad]).any() and torch.equal(y[~bad], clean[~bad])


def test_empty_sides():
    f = fqa()
    for fmt in R.FORMATS:
        a, e = R.random_microscaled(5, 64, fmt, 1), R.random_microscaled(0, 64, fmt, 2)
        assert f.mx_matmul(e, a).shape == (0, 5) and f.mx_matmul(a, e).shape == (5, 0)


@pytest.mark.parametrize("M", [1, 100, 1500, 3000])
def test_the_same_call_gives_the_same_bits(M):
    f = fqa()
    a, b = R.random_microscaled(M, 4096, "nvfp4", 1), R.random_microscaled(1030, 4096, "nvfp4", 2)
    first = f.mx_matmul(a, b)
    for _ in range(5):
        assert torch.equal(first, f.mx_matmul(a, b))


def test_two_streams_at_once_and_replayed_graphs():
    f = fqa()
    sizes = ((1, 4096, 4096), (100, 1000, 2048), (2500, 1500, 1024))
    ops = [(R.random_microscaled(M, K, "nvfp4", 1), R.random_microscaled(N, K, "nvfp4", 2)) for M, N, K in sizes]
    want = [f.mx_matmul(a, b) for a, b in ops]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[f.mx_matmul(a, b, stream=st) for _ in range(10) for a, b in ops] for st in s]
    torch.cuda.synchronize()
    for side in got:
        for i, y in enumerate(side):
            assert torch.equal(y, want[i % 3])
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([f.mx_matmul(a, b) for a, b in ops])
        graphs.append(g)
    for st, g in zip(s, graphs):
        with torch.cuda.stream(st):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(y, w) for y, w in zip(o, want))
    assert f.fqa_debug_status()[0] == f.FQA_OK


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_a_block_up_to_its_attention(fmt):
    """Residual stream -> norm and quantization -> QKV projection -> positions on
    the packed result's views -> FP8 attention, against the same chain in 64 bits
    on the library's own codes where codes decide."""
    f = fqa()
    B, N, H, K = 1, 200, 2, 384
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(N, K, device="cuda", generator=g).bfloat16()
    r = torch.randn(N, K, device="cuda", generator=g).bfloat16()
    wn = (1 + 0.1 * torch.randn(K, device="cuda", generator=g)).bfloat16()
    w = f.mx_quantize((torch.randn(3 * H * 128, K, device="cuda", generator=g) / K ** 0.5).bfloat16(), fmt)
    y, h = f.mx_rms_norm(x, wn, fmt, residual=r)
    packed = f.mx_matmul(y, w)
    ref, mag = reference(y, w, None)
    assert ((packed.double() - ref).abs() <= bound(ref, mag, K, torch.bfloat16)).all()
    q, k, v = (packed.view(B, N, 3, H, 128)[:, :, i].transpose(1, 2) for i in range(3))
    qw = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos = torch.stack([torch.arange(N) // 100, torch.arange(N) // 10 % 10, torch.arange(N) % 10], 1).int().cuda()
    rot = f.Rotary(pos, (16, 56, 56), q_weight=qw, k_weight=qw)
    out = f.fp8_attention(q, k, v.contiguous(), f.softmax_scale(), f.FQA_OUT_F32, rot=rot)
    q64, k64 = (torch.from_numpy(R.rotary(t, pos, (16, 56, 56), weight=qw)).cuda() for t in (q, k))
    p = torch.softmax(q64 @ k64.transpose(2, 3) * f.softmax_scale(), -1)
    want = p @ v.double()
    # E4M3 operands (2^-4 each on q, k, v, p): a loose bound that a wrong layout,
    # head or position breaks by far
    rel = (out.double() - want).norm() / want.norm()
    assert rel < 4 * 2.0 ** -4
    assert f.fqa_debug_status()[0] == f.FQA_OK


def test_every_row_count_around_the_tiles():
    """1 to 300 rows against one set of weights: each row is the row that the
    whole product has (the split of K, and with it the sum's order, may differ
    with the row count, so to the sums' rounding)."""
    f = fqa()
    K, N = 2080, 200
    a, b = R.random_microscaled(300, K, "nvfp4", 1, wide=True), R.random_microscaled(N, K, "nvfp4", 2, wide=True)
    y, mag = reference(a, b, None)
    lim = bound(y, mag, K, torch.float32)
    x = f.mx_dequantize(a, 1)
    for M in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300):
        part = f.Microscaled(a.codes[:M].contiguous(), a.scales[: -(-M // 128)].contiguous(),
                             a.row_scale[:M].contiguous(), K, "nvfp4")
        err = (f.mx_matmul(part, b, out_dtype=1).double() - y[:M]).abs()
        assert (err <= lim[:M]).all(), M
    assert x.shape == (300, K)


def test_a_chain_without_waiting():
    """Norm, product, quantization, product and the way back over the same
    buffers again and again, nothing waited for: launches overlap with the end of
    the one before, and have to give what they give one at a time."""
    f = fqa()
    g = torch.Generator(device="cuda").manual_seed(1)
    M, K, N = 500, 1024, 768
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    up = f.mx_quantize(torch.randn(N, K, device="cuda", generator=g).bfloat16() / 32, "nvfp4")
    down = f.mx_quantize(torch.randn(K, N, device="cuda", generator=g).bfloat16() / 28, "nvfp4")

    def run(wait):
        h = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        step = x.clone()
        q, m = f.alloc_microscaled(M, K, "nvfp4", "cuda"), f.alloc_microscaled(M, N, "nvfp4", "cuda")
        mid = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        for _ in range(60):
            f.mx_rms_norm(step, w, "nvfp4", residual=h, residual_out=h, out=q)
            if wait:
                torch.cuda.synchronize()
            f.mx_matmul(q, up, out=mid)
            if wait:
                torch.cuda.synchronize()
            f.mx_quantize(mid, "nvfp4", out=m)
            if wait:
                torch.cuda.synchronize()
            f.mx_matmul(m, down, out=step)
            if wait:
                torch.cuda.synchronize()
        return h.clone(), step.clone()
    want, got = run(True), run(False)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and torch.isfinite(want[0]).all()


def test_results_beyond_two_to_the_31():
    f = fqa()
    M, N = 70001, 32000                       # 2.24e9 results
    a, b = R.random_microscaled(M, 32, "mxfp8", 1), R.random_microscaled(N, 32, "mxfp8", 2)
    y = f.mx_matmul(a, b)
    last = f.Microscaled(a.codes[-113:].contiguous(), a.scales[-1:].contiguous(), None, 32, "mxfp8")
    assert M - 113 == a.scales[:-1].shape[0] * 128
    assert torch.equal(y[-113:], f.mx_matmul(last, b))
    assert torch.equal(y[:128], f.mx_matmul(f.Microscaled(a.codes[:128], a.scales[:1], None, 32, "mxfp8"), b))
