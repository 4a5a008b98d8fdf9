"""Cases of the operators around the attention call: rotary positions over
several axes, microscaled quantization, the RMS norm that feeds it, and the
block-scaled product.

`own` chooses between the plain form (elementary torch operations) and the
library's calls.  Formats: "mxfp8" (E4M3 elements, a power of two per 32),
"mxfp4" (E2M1, a power of two per 32), "nvfp4" (E2M1, an E4M3 scale per 16 and
a binary32 scale per row, a power of two where it is chosen here)."""

import math

import numpy as np
import torch

own = False

HEAD_DIM = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
PER_BYTE = {"mxfp8": 1, "mxfp4": 2, "nvfp4": 2}


def listed():
    return [
        # one new token per sequence of a small batch: only latency counts
        dict(name="rotary 1 token", op="rotary", B=4, N=1, Hq=24, Hk=24, axes="16,56,56", split=False, shared=False,
             norm=True, fractional=False, inverse=False, dtype="bf16"),
        # one block's Q and K of a 1024 x 1024 image with its text (N = 4608, 24 heads), normalized per head
        dict(name="rotary image 4608", op="rotary", B=1, N=4608, Hq=24, Hk=24, axes="16,56,56", split=False,
             shared=False, norm=True, fractional=False, inverse=False, dtype="bf16"),
        # a video-sized pair of sequences, fractional times, shared key heads, an odd length, rotated back
        dict(name="rotary video 16895", op="rotary", B=2, N=16895, Hq=24, Hk=8, axes="32,48,48", split=True, shared=True,
             norm=False, fractional=True, inverse=True, dtype="bf16"),
        # weights of a projection, quantized once when they are loaded
        dict(name="quantize nvfp4 weights", op="quantize", fmt="nvfp4", M=12288, K=4096, dtype="bf16"),
        # a caption's activations: few rows, an odd width, half precision
        dict(name="quantize mxfp4 77", op="quantize", fmt="mxfp4", M=77, K=2001, dtype="f16"),
        # a single token's residual step
        dict(name="norm 1 token", op="norm", fmt="mxfp8", M=1, K=4096, residual=True, dtype="bf16"),
        # the residual stream of one block, image and context image (N = 8704)
        dict(name="norm 8704", op="norm", fmt="mxfp8", M=8704, K=4096, residual=True, dtype="bf16"),
        # a wide, ragged binary32 stream into 4 bits
        dict(name="norm f32 1023", op="norm", fmt="nvfp4", M=1023, K=5100, residual=True, dtype="f32"),
        # one token against a square projection: the weights' bytes are all that counts
        dict(name="product 1 token", op="product", fmt="nvfp4", M=1, N=4096, K=4096, bias=False, out="bf16"),
        # a caption through an odd-sized projection, kept in binary32
        dict(name="product 77", op="product", fmt="mxfp4", M=77, N=2111, K=4128, bias=True, out="f32"),
        # a 1024 x 1024 image's tokens in 8 bits
        dict(name="product mxfp8 4608", op="product", fmt="mxfp8", M=4608, N=4096, K=4096, bias=True, out="bf16"),
        # the QKV projection of 8704 tokens in 4 bits: the largest product
        dict(name="product nvfp4 8704", op="product", fmt="nvfp4", M=8704, N=12288, K=4096, bias=False, out="bf16"),
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotary", "quantize", "norm", "product"))
    if op == "rotary":
        B = rng.choice((1, 1, 2, 3, 4))
        Hq = rng.choice((1, 2, 8, 16, 24, 32))
        Hk = rng.choice([h for h in (1, 2, 4, 8, 16, 24, 32) if Hq % h == 0])
        most = max(1, 2 * 24 * 16896 * 2 // (B * (Hq + Hk)))
        split = rng.random() < 0.5
        axes = rng.choice(("128", "64,64", "16,56,56", "32,48,48", "16,24,24", "8,40,40,40") if split else
                          ("128", "64,64", "16,56,56", "32,48,48", "44,42,42", "10,20,30", "2,4"))
        return dict(op="rotary", B=B, N=_spread(rng, 1, min(65536, most)), Hq=Hq, Hk=Hk, axes=axes, split=split,
                    shared=rng.random() < 0.5, norm=rng.random() < 0.5, fractional=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
    fmt = rng.choice(("mxfp8", "mxfp4", "nvfp4"))
    if op in ("quantize", "norm"):
        K = _spread(rng, 32, 20000)
        K = K if rng.random() < 0.4 else max(32, K // 64 * 64)
        case = dict(op=op, fmt=fmt, M=_spread(rng, 1, max(1, min(16384, 12288 * 4096 // K))), K=K)
        if op == "norm":
            case["residual"] = rng.random() < 0.7
        return dict(case, dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
    K, N = _spread(rng, 32, 16384), _spread(rng, 32, 16384)
    if rng.random() < 0.6:
        K, N = max(32, K // 32 * 32), max(32, N // 64 * 64)
    return dict(op="product", fmt=fmt, M=_spread(rng, 1, max(1, min(8704, 8704 * 12288 * 4096 // (N * K)))), N=N, K=K,
                bias=rng.random() < 0.5, out=rng.choice(("bf16", "bf16", "f16", "f32")))


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activations(g, rows, cols):
    """Normal values with a few loud columns and rows of different loudness."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    loud = torch.where(torch.rand(1, cols, device="cuda", generator=g) < 0.01, 20.0, 1.0)
    return x * loud * torch.exp(torch.randn(rows, 1, device="cuda", generator=g))


def _padded(cols):
    return -(-cols // 32) * 32


def _tiles(scale_bytes, rows):
    """Row-major scale bytes [rows, blocks] in tiles of 128 rows x 4 blocks: [rows/128, blocks/4, 32, 4, 4],
    row r of a tile at [r % 32, r / 32]."""
    mt, kt = -(-rows // 128), -(-scale_bytes.shape[1] // 4)
    full = torch.zeros(mt * 128, kt * 4, dtype=torch.uint8, device=scale_bytes.device)
    full[:rows, : scale_bytes.shape[1]] = scale_bytes
    return full.view(mt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous()


def _packed(x, fmt):
    """(codes, scale tiles, row scales or None) of x as the formats hold them."""
    elements, scale_bytes, _, row = _coded(x.float(), fmt)
    rows = x.shape[0]
    if fmt == "mxfp8":
        codes = elements.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        mag = elements.abs()
        code = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8)
        code = code + 8 * torch.signbit(elements).to(torch.uint8)
        codes = code[:, 0::2] + 16 * code[:, 1::2]
    return codes.contiguous(), _tiles(scale_bytes, rows), row


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "rotary":
        B, N, Hq, Hk = case["B"], case["N"], case["Hq"], case["Hk"]
        dt = DTYPES[case["dtype"]]
        # the packed output of a QKV projection: [B, N, Hq + 2 Hk, 128], Q and K heads first
        packed = torch.randn(B, N, Hq + 2 * Hk, HEAD_DIM, device="cuda", generator=g)
        packed = (packed * torch.exp(0.5 * torch.randn(HEAD_DIM, device="cuda", generator=g))).to(dt)
        n_axes = len(case["axes"].split(","))
        # text tokens at the origin, then a grid of images: time slowest, width fastest; a sequence starts at an offset
        text = min(512, N // 8)
        cell = (torch.arange(N, device="cuda") - text).clamp(min=0)
        side = max(1, min(128, math.isqrt(max(1, N - text))))
        grid = torch.stack([cell // (side * side), cell // side % side, cell % side, cell // 7], 1)[:, :n_axes]
        if n_axes == 1:
            grid = torch.arange(N, device="cuda")[:, None]
        start = torch.randint(0, 1000, (B, 1, n_axes), device="cuda", generator=g)
        positions = grid[None] + start * (torch.arange(N, device="cuda") >= text)[None, :, None]
        positions = positions.float() * 0.625 if case["fractional"] else positions.to(torch.int32)
        weights = [None, None]
        if case["norm"]:
            weights = [(1 + 0.2 * torch.randn(HEAD_DIM, device="cuda", generator=g)).to(dt) for _ in range(2)]
        return dict(case=case, axes=tuple(map(int, case["axes"].split(","))), q=packed[:, :, :Hq].transpose(1, 2),
                    k=packed[:, :, Hq : Hq + Hk].transpose(1, 2),
                    positions=positions.contiguous(), q_weight=weights[0], k_weight=weights[1])
    if case["op"] == "product":
        a = _activations(g, case["M"], case["K"]).to(torch.bfloat16)
        b = (torch.randn(case["N"], case["K"], device="cuda", generator=g) / math.sqrt(case["K"])).to(torch.bfloat16)
        a, b = _packed(a, case["fmt"]), _packed(b, case["fmt"])
        if case["fmt"] == "nvfp4":  # weights under a calibrated scale of their own, which is no power of two
            b = (*b[:2], b[2] * (0.5 + torch.rand(1, device="cuda", generator=g)))
        state = dict(case=case, a=a, b=b, bias=None)
        if case["bias"]:
            state["bias"] = torch.randn(case["N"], device="cuda", generator=g)
        return state
    dt = DTYPES[case["dtype"]]
    state = dict(case=case, x=_activations(g, case["M"], case["K"]).to(dt))
    if case["op"] == "norm":
        state["weight"] = (1 + 0.2 * torch.randn(case["K"], device="cuda", generator=g)).to(dt)
        state["residual"] = _activations(g, case["M"], case["K"]).to(dt) if case["residual"] else None
    return state


# --------------------------------------------------------------- plain form

def _round_e2m1(x):
    mag = x.abs().clamp(max=6.0)
    mag = torch.where(mag < 2, torch.round(mag * 2) / 2, torch.where(mag < 4, torch.round(mag), torch.round(mag / 2) * 2))
    return torch.copysign(mag, x)


def _round_e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()


def _power_of_two(e):
    """2^e in binary32 for whole -127 <= e <= 127, exactly."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).int().view(torch.float32)


def _smallest_power(amax, largest):
    """The smallest whole e >= -127 with amax <= largest * 2^e."""
    mantissa, exponent = torch.frexp(amax)
    part, top = math.frexp(largest)
    return torch.where(amax > 0, exponent - top + (mantissa > part).int(), -127).clamp(min=-127)


def _coded(x, fmt):
    """(elements as values, scale bytes, scale values per block, row scales or None) of binary32 rows."""
    rows, cols = x.shape
    block = BLOCK[fmt]
    x = torch.nn.functional.pad(x, (0, _padded(cols) - cols)).view(rows, -1, block)
    amax = x.abs().amax(2)
    if fmt == "nvfp4":
        e = _smallest_power(amax.amax(1), 2688.0).clamp(min=-126)[:, None]
        amax, x = amax * _power_of_two(-e), x * _power_of_two(-e)[:, :, None]
        scale = _round_e4m3(amax / torch.full_like(amax, 6.0))  # a true division: by a number, torch multiplies with its reciprocal
        elements = _round_e2m1(torch.where(scale[:, :, None] > 0, x / scale[:, :, None], 0.0))
        return elements.view(rows, -1), scale.to(torch.float8_e4m3fn).view(torch.uint8), scale, _power_of_two(e)[:, 0]
    e = _smallest_power(amax, 448.0 if fmt == "mxfp8" else 6.0)
    scaled = x * _power_of_two(-e)[:, :, None]
    elements = _round_e4m3(scaled) if fmt == "mxfp8" else _round_e2m1(scaled)
    return elements.view(rows, -1), (e + 127).to(torch.uint8), _power_of_two(e), None


def _stands_for(x, fmt):
    """The values that the codes of x stand for, in binary32, without the padding."""
    elements, _, scale, row = _coded(x, fmt)
    values = elements.view(x.shape[0], -1, BLOCK[fmt]) * scale[:, :, None]
    values = values if row is None else values * row[:, None, None]
    return values.view(x.shape[0], -1)[:, : x.shape[1]]


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _unpacked(packed, fmt, dtype=torch.float32):
    """The values of held codes, padding included."""
    codes, tiles, row = packed
    if fmt == "mxfp8":
        elements = codes.view(torch.float8_e4m3fn).to(dtype)
    else:
        table = torch.tensor(E2M1, dtype=dtype, device=codes.device)
        elements = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], 2).flatten(1)
    rows, block = codes.shape[0], BLOCK[fmt]
    flat = tiles.permute(0, 3, 2, 1, 4).reshape(-1, 4 * tiles.shape[1])[:rows, : elements.shape[1] // block]
    if fmt == "nvfp4":
        scale = flat.contiguous().view(torch.float8_e4m3fn).to(dtype)
    else:
        scale = _power_of_two(flat.int() - 127).to(dtype)
    values = (elements.view(rows, -1, block) * scale[:, :, None]).view(rows, -1)
    return values if row is None else values * row.to(dtype)[:, None]


def _frequencies(axes, case):
    """Per pair: its axis and its angle per position, in 64 bits, in the order of the pairs."""
    axes = torch.tensor(axes, device="cuda")
    axis = torch.repeat_interleave(torch.arange(len(axes), device="cuda"), axes // 2)
    first = (torch.cumsum(axes, 0) - axes)[axis] // 2
    pair = torch.arange(len(axis), device="cuda")
    if case["shared"]:
        return axis, 10000.0 ** (-2.0 * pair.double() / axes.sum())
    return axis, 10000.0 ** (-2.0 * (pair - first).double() / axes[axis])


def _rotated(x, weight, cos, sin, case):
    dt = x.dtype
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    pairs = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if case["split"]:
        x0, x1, rest = x[..., :pairs], x[..., pairs : 2 * pairs], x[..., 2 * pairs :]
        return torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos, rest], -1).to(dt)
    x0, x1, rest = x[..., 0 : 2 * pairs : 2], x[..., 1 : 2 * pairs : 2], x[..., 2 * pairs :]
    both = torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)
    return torch.cat([both, rest], -1).to(dt)


def run(state):
    case = state["case"]
    if own:
        import quantized_fp8_attention_b200 as fqa
        codes = {"bf16": fqa.FQA_OUT_BF16, "f32": fqa.FQA_OUT_F32, "f16": fqa.FQA_OUT_F16}
        if case["op"] == "rotary":
            rot = fqa.Rotary(state["positions"], state["axes"], split=case["split"],
                             shared=case["shared"], q_weight=state["q_weight"], k_weight=state["k_weight"])
            q, k = fqa.rotary(state["q"], state["k"], rot, inverse=case["inverse"])
            return {"q": q, "k": k}
        if case["op"] == "product":
            a, b = (fqa.Microscaled(*state[x], case["K"], case["fmt"]) for x in "ab")
            return {"y": fqa.mx_matmul(a, b, bias=state["bias"], out_dtype=codes[case["out"]])}
        if case["op"] == "quantize":
            return {"values": fqa.mx_dequantize(fqa.mx_quantize(state["x"], case["fmt"]))}
        y, h = fqa.mx_rms_norm(state["x"], state["weight"], case["fmt"], residual=state["residual"])
        out = {"values": fqa.mx_dequantize(y)}
        return out if h is None else dict(out, residual=h)
    if case["op"] == "rotary":
        axis, frequency = _frequencies(state["axes"], case)
        angle = state["positions"].double()[..., axis] * frequency
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float() * (-1 if case["inverse"] else 1)
        return {"q": _rotated(state["q"], state["q_weight"], cos, sin, case),
                "k": _rotated(state["k"], state["k_weight"], cos, sin, case)}
    if case["op"] == "product":
        y = _unpacked(state["a"], case["fmt"]) @ _unpacked(state["b"], case["fmt"]).T
        y = y if state["bias"] is None else y + state["bias"]
        return {"y": y.to(DTYPES[case["out"]])}
    if case["op"] == "quantize":
        return {"values": _stands_for(state["x"].float(), case["fmt"]).to(torch.bfloat16)}
    h = state["x"].float() if state["residual"] is None else state["x"].float() + state["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * state["weight"].float()
    out = {"values": _stands_for(y, case["fmt"]).to(torch.bfloat16)}
    return out if state["residual"] is None else dict(out, residual=h.to(state["x"].dtype))


# ---------------------------------------------------------------- the work

def work(case):
    if case["op"] == "rotary":
        elements = case["B"] * case["N"] * (case["Hq"] + case["Hk"]) * HEAD_DIM
        n_axes = len(case["axes"].split(","))
        return {"bytes": 2 * BYTES[case["dtype"]] * elements + 4 * case["B"] * case["N"] * n_axes,
                "flops": elements * (7 if case["norm"] else 3)}
    if case["op"] == "product":
        M, N, Kp, fmt = case["M"], case["N"], _padded(case["K"]), case["fmt"]
        held = Kp // PER_BYTE[fmt] + Kp // BLOCK[fmt] + (4 if fmt == "nvfp4" else 0)
        return {"bytes": (M + N) * held + M * N * BYTES[case["out"]] + (4 * N if case["bias"] else 0),
                "flops": 2 * M * N * case["K"]}
    elements = case["M"] * case["K"]
    if case["op"] == "quantize":
        return {"bytes": elements * (BYTES[case["dtype"]] + 2), "flops": 4 * elements}
    streams = 3 if case["residual"] else 1
    return {"bytes": elements * (streams * BYTES[case["dtype"]] + 2), "flops": 8 * elements}


# ---------------------------------------------------- in 64 bits, from the definitions

def _nearest(x, table):
    """The nearest entry of an ascending table of non-negative values to |x|, ties to the even index, with x's sign."""
    table = torch.tensor(table, dtype=torch.float64, device=x.device)
    mid = (table[1:] + table[:-1]) / 2
    mag = x.abs()
    i = torch.searchsorted(mid, mag)
    tie = (i < len(mid)) & (mid[i.clamp(max=len(mid) - 1)] == mag) & (i % 2 == 1)
    return torch.where(x < 0, -1.0, 1.0) * table[i + tie.long()]


def _two64(power):
    """2^power in binary64 for whole powers in its normal range, put together from its exponent bits."""
    return ((power.long() + 1023) << 52).view(torch.float64)


def _power64(top, largest):
    """The smallest power of at least -127 whose `largest` multiple reaches top, found from the logarithm's neighbours."""
    power = torch.ceil(torch.log2(torch.where(top > 0, top, 1e-100) / largest)).clamp(min=-127)
    power = torch.where((largest * _two64(power - 1) >= top) & (power > -127), power - 1, power)
    return torch.where(largest * _two64(power) < top, power + 1, power)


def _quantized64(x, fmt):
    e4m3 = [m * 2.0**-9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    rows, cols = x.shape
    full = torch.zeros(rows, _padded(cols), dtype=torch.float64, device=x.device)
    full[:, :cols] = x
    blocks = full.view(rows, -1, BLOCK[fmt])
    top = blocks.abs().max(2, keepdim=True).values
    if fmt == "nvfp4":
        row = _two64(_power64(blocks.abs().amax((1, 2), keepdim=True), 2688.0).clamp(min=-126))
        scale = _nearest(top / (6 * row), e4m3)
        step = scale * row
        values = step * _nearest(blocks / torch.where(step > 0, step, 1.0), E2M1[:8]) * (step > 0)
    else:
        table = e4m3 if fmt == "mxfp8" else E2M1[:8]
        step = _two64(_power64(top, table[-1]))
        values = step * _nearest(blocks / step, table)
    return values.reshape(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        axes = [int(a) for a in case["axes"].split(",")]
        out, total, angles, done = {}, sum(axes), [], 0
        for a, width in enumerate(axes):
            index = np.arange(width // 2) + (done // 2 if case["shared"] else 0)
            f = torch.from_numpy(np.power(10000.0, -2.0 * index / (total if case["shared"] else width))).cuda()
            angles.append(s["positions"][..., a : a + 1].double() * f)
            done += width
        angle = torch.cat(angles, -1)[:, None]
        unit = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)
        for name in "qk":
            x = s[name].double()
            w = s[name + "_weight"]
            if w is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / HEAD_DIM + 1e-6) * w.double()
            first = list(range(total // 2)) if case["split"] else list(range(0, total, 2))
            second = list(range(total // 2, total)) if case["split"] else list(range(1, total, 2))
            z = torch.complex(x[..., first], x[..., second]) * unit
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            out[name] = y
        return out
    if case["op"] == "product":
        a, b = (_values64(*s[x], case["fmt"]) for x in "ab")
        y = torch.einsum("mk,nk->mn", a, b)
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    if case["op"] == "quantize":
        return {"values": _quantized64(s["x"].double(), case["fmt"])}
    h = s["x"].double()
    if s["residual"] is not None:
        h = h + s["residual"].double()
    y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["K"] + 1e-6) * s["weight"].double()
    out = {"values": _quantized64(y, case["fmt"])}
    return out if s["residual"] is None else dict(out, residual=h)


def _values64(codes, tiles, row, fmt):
    """The held values in 64 bits, each format's bits taken apart by arithmetic."""
    c = codes.long()
    if fmt == "mxfp8":
        e, m = c // 8 % 16, c % 8
        values = torch.where(e > 0, (8 + m) * _two64(e - 10), m * 2.0**-9) * (1 - 2 * (c // 128))
    else:
        c = torch.stack([c % 16, c // 16], 2).view(c.shape[0], -1)
        e, m = c // 2 % 4, c % 2
        values = torch.where(e > 0, (2 + m) * _two64(e - 2), m * 0.5) * (1 - 2 * (c // 8))
    r = torch.arange(codes.shape[0], device=codes.device)[:, None]
    j = (torch.arange(values.shape[1], device=codes.device) // BLOCK[fmt])[None]
    held = tiles[r // 128, j // 4, r % 32, r // 32 % 4, j % 4].long()
    if fmt == "nvfp4":
        scale = torch.where(held >= 8, (8 + held % 8) * _two64(held // 8 - 10), held * 2.0**-9)
        return values * scale * row.double()[:, None]
    return values * _two64(held - 127)
