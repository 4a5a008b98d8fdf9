"""Plain 64-bit implementations of the operators around the attention call, on
the CPU: microscaled rows, RMS norm, product, rotary positions.  Written from the
definitions in include/fqa.h, element by element where that stays quick."""

from __future__ import annotations

import numpy as np
import torch

E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
FORMATS = tuple(BLOCK)


def nearest(x, table):
    """Codes (magnitude's index) of the nearest table entries, ties to the even
    index, saturating; x in binary64."""
    mag = np.abs(x)
    mid = (table[1:] + table[:-1]) / 2
    i = np.searchsorted(mid, mag, side="left")           # mid[i-1] < mag <= mid[i]
    j = np.minimum(i, len(mid) - 1)
    return i + ((i < len(mid)) & (mid[j] == mag) & (i % 2 == 1))


def smallest_power(amax, largest, low):
    """The smallest whole e >= low with amax <= largest 2^e."""
    e = np.full(amax.shape, low)
    while True:
        small = amax > largest * 2.0 ** e
        if not small.any():
            return e
        # far below: jump by the ratio's exponent, then step
        ratio = np.where(small, amax / (largest * 2.0 ** e), 1.0)
        e = e + np.where(small, np.maximum(1, np.floor(np.log2(ratio)).astype(int) - 1), 0)


def quantize(x, fmt):
    """binary64 rows -> (codes as magnitude index + sign bit, scale bytes [M, blocks],
    row scales or None), all arrays; non-finite blocks and rows by the rule."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    kp = -(-K // 32) * 32
    full = np.zeros((M, kp))
    full[:, :K] = x
    b = full.reshape(M, -1, BLOCK[fmt])
    finite = np.isfinite(b).all(2)
    if fmt == "nvfp4":
        finite = np.broadcast_to(finite.all(1, keepdims=True), finite.shape)
    b = np.where(finite[:, :, None], b, 0.0)
    amax = np.abs(b).max(2)
    if fmt == "nvfp4":
        e = smallest_power(amax.max(1), 2688.0, -126)
        row = np.where(finite[:, 0], 2.0 ** e, np.nan)
        y = b / (2.0 ** e)[:, None, None]
        # the quotient by 6 is rounded to binary32 before it becomes a scale
        s = nearest(((amax / (2.0 ** e)[:, None]).astype(np.float32) / np.float32(6)).astype(np.float64), E4M3)
        scale = E4M3[s]
        q = np.where(scale[:, :, None] > 0, y / np.where(scale > 0, scale, 1.0)[:, :, None], 0.0)
        table, bytes_ = E2M1, s.astype(np.uint8)
    else:
        row = None
        table = E4M3 if fmt == "mxfp8" else E2M1
        e = smallest_power(amax, table[-1], -127)
        q = b / (2.0 ** e)[:, :, None]
        bytes_ = np.where(finite, e + 127, 255).astype(np.uint8)
    sign = 128 if fmt == "mxfp8" else 8
    codes = nearest(q, table) + np.where(np.signbit(q), sign, 0)
    return codes.reshape(M, kp).astype(np.uint8), bytes_, row


def untile(scales, M, blocks):
    """Scale tiles (a tensor [mt, kt, 32, 4, 4]) -> row-major bytes [M, blocks]."""
    t = scales.cpu().numpy()
    r, j = np.arange(M)[:, None], np.arange(blocks)[None, :]
    return t[r // 128, j // 4, r % 32, r // 32 % 4, j % 4]


def held(q):
    """A Microscaled's (codes, scale bytes, row scales) in the form of quantize()."""
    codes = q.codes.cpu().numpy()
    if q.fmt != "mxfp8":
        codes = np.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1)
    M = codes.shape[0]
    return codes, untile(q.scales, M, codes.shape[1] // BLOCK[q.fmt]), (
        None if q.row_scale is None else q.row_scale.cpu().numpy().astype(np.float64))


def values(codes, bytes_, row, fmt, cols=None):
    """What codes stand for, in binary64 (NaN where a scale says so)."""
    table = E4M3 if fmt == "mxfp8" else E2M1
    bits = 128 if fmt == "mxfp8" else 8
    v = np.where(codes & bits, -1.0, 1.0) * table[np.minimum(codes % bits, len(table) - 1)]
    M = codes.shape[0]
    if fmt == "nvfp4":
        scale = E4M3[bytes_ & 127]
    else:
        scale = np.where(bytes_ == 255, np.nan, 2.0 ** (bytes_.astype(int) - 127.0))
    v = (v.reshape(M, -1, BLOCK[fmt]) * scale[:, :, None]).reshape(M, -1)
    if row is not None:
        v = v * np.asarray(row, dtype=np.float64)[:, None]
    return v if cols is None else v[:, :cols]


def rms_norm(x, weight, residual, eps):
    """(y, h) in binary64."""
    h = x.double().cpu().numpy()
    if residual is not None:
        h = h + residual.double().cpu().numpy()
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight.double().cpu().numpy()
    return y, h


def rotary(x, positions, axes, theta=10000.0, split=False, shared=False, inverse=False, weight=None, eps=1e-6):
    """x [B,H,N,128] -> binary64 [B,H,N,128], pair by pair."""
    x = x.double().cpu().numpy()
    B, H, N, d = x.shape
    if weight is not None:
        x = x / np.sqrt((x * x).mean(3, keepdims=True) + eps) * weight.double().cpu().numpy()
    pos = positions.double().cpu().numpy()
    pos = np.broadcast_to(pos if pos.ndim == 3 else pos[None], (B, N, len(axes)))
    y, D, j = x.copy(), sum(axes), 0
    for a, width in enumerate(axes):
        for i in range(width // 2):
            angle = pos[:, None, :, a] * theta ** -(2.0 * j / D if shared else 2.0 * i / width)
            c, s = np.cos(angle), np.sin(angle) * (-1 if inverse else 1)
            u, v = (j, D // 2 + j) if split else (2 * j, 2 * j + 1)
            y[..., u] = x[..., u] * c - x[..., v] * s
            y[..., v] = x[..., u] * s + x[..., v] * c
            j += 1
    return y


def random_microscaled(M, K, fmt, seed, device="cuda", wide=False):
    """A Microscaled of random codes and moderate random scales, built here.
    `wide`: row scales that are no powers of two."""
    import quantized_fp8_attention_b200 as fqa
    g = np.random.default_rng(seed)
    kp = -(-K // 32) * 32
    blocks = kp // BLOCK[fmt]
    if fmt == "mxfp8":
        codes = g.integers(0, 256, (M, kp), dtype=np.uint8)
        codes = np.where((codes & 127) == 127, 0, codes).astype(np.uint8)     # no NaN codes
    else:
        codes = g.integers(0, 16, (M, kp), dtype=np.uint8)
    codes[:, K:] = 0
    bytes_ = g.integers(0x30, 0x48, (M, blocks)) if fmt == "nvfp4" else g.integers(120, 130, (M, blocks))
    row = None
    if fmt == "nvfp4":
        row = (g.uniform(0.5, 2.0, M) if wide else 2.0 ** g.integers(-4, 5, M)).astype(np.float32)
    mt, words = -(-M // 128), -(-blocks // 4)
    tiles = g.integers(0, 256, (mt, words, 32, 4, 4), dtype=np.uint8)          # rows past M: anything
    r, j = np.arange(M)[:, None], np.arange(words * 4)[None, :]
    full = np.zeros((M, words * 4), dtype=np.uint8)
    full[:, :blocks] = bytes_
    tiles[r // 128, j // 4, r % 32, r // 32 % 4, j % 4] = full
    packed = codes if fmt == "mxfp8" else codes[:, 0::2] | (codes[:, 1::2] << 4)
    put = lambda t: torch.from_numpy(np.ascontiguousarray(t)).to(device)
    return fqa.Microscaled(put(packed), put(tiles), None if row is None else put(row), K, fmt)
