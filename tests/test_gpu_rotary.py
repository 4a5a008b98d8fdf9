"""Rotary positions on the GPU against the 64-bit reference."""

import numpy as np
import pytest
import torch

from tests import block_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def fqa():
    import quantized_fp8_attention_b200 as f
    return f


def close(got, want, x, weight, norm_rows):
    """cos and sin are off by at most 2^-25 turns (the reduced angle's rounding,
    2 pi 2^-25 = 2^-22.35) and 2^-23 of sincospif, two products and a sum round
    by 2^-24 each: |dy| <= 0.51 2^-20 (|x0| + |x1|) <= 1.02 2^-20 max |y| over the
    row (|x0| + |x1| <= 2 max), held to 1.5 2^-20.  The norm adds at most 16
    roundings, halved, rsqrtf's two units and two products, under 2^-20 again.
    Then one rounding to the type."""
    t = got.dtype
    top = np.abs(want).max(-1, keepdims=True)
    tol = (2.0 ** -19 if norm_rows else 2.0 ** -20) * 1.5 * top + torch.finfo(t).eps / 2 * np.abs(want)
    if t == torch.float16:
        tol = tol + 2.0 ** -25
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err - tol).max())


def run(B, N, Hq, Hk, axes, dt="bf16", split=False, shared=False, norm=False, inverse=False, fractional=False,
        batched=True, top=2000, seed=0, view="tokens"):
    f = fqa()
    g = torch.Generator(device="cuda").manual_seed(seed)
    H = Hq + Hk + 1
    if view == "tokens":
        packed = torch.randn(B, N, H, 128, device="cuda", generator=g).to(DT[dt])
        q, k = packed[:, :, :Hq].transpose(1, 2), packed[:, :, Hq:Hq + Hk].transpose(1, 2)
    elif view == "heads":
        q = torch.randn(B, Hq, N, 128, device="cuda", generator=g).to(DT[dt])
        k = torch.randn(B, Hk, N, 128, device="cuda", generator=g).to(DT[dt])
    else:                                     # rows off every vector boundary
        packed = torch.randn(B, N, H * 130 + 1, device="cuda", generator=g).to(DT[dt])[:, :, 1:]
        packed = packed.unflatten(2, (H, 130))[..., 1:129]
        q, k = packed[:, :, :Hq].transpose(1, 2), packed[:, :, Hq:Hq + Hk].transpose(1, 2)
    shape = (B, N, len(axes)) if batched else (N, len(axes))
    pos = torch.randint(-top, top, shape, device="cuda", generator=g, dtype=torch.int32)
    if fractional:
        pos = pos.float() * 0.37
    w = [(1 + 0.3 * torch.randn(128, device="cuda", generator=g)).to(DT[dt]) if norm else None for _ in range(2)]
    rot = f.Rotary(pos, axes, split=split, shared=shared, q_weight=w[0], k_weight=w[1])
    qo, ko = f.rotary(q, k, rot, inverse=inverse)
    for got, x, wt in ((qo, q, w[0]), (ko, k, w[1])):
        assert got.is_contiguous() and got.shape == x.shape and got.dtype == x.dtype
        if x.numel():
            close(got, R.rotary(x, pos, axes, split=split, shared=shared, inverse=inverse, weight=wt), x, wt, norm)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("axes", [(128,), (64, 64), (16, 56, 56), (8, 40, 40, 40), (16, 24, 24), (16,)])
def test_axes_and_pairings(axes, split, shared):
    run(2, 21, 3, 2, axes, split=split, shared=shared)
    run(1, 5, 2, 1, axes, split=split, shared=shared, norm=True, dt="f32")


@pytest.mark.parametrize("axes", [(2, 4), (10, 20, 30), (2,), (6, 6, 6, 6)])
def test_widths_that_are_no_multiple_of_a_vector(axes):
    run(1, 19, 2, 2, axes, dt="f16")
    run(1, 19, 2, 2, axes, norm=True)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("view", ["tokens", "heads", "odd"])
@pytest.mark.parametrize("split", [False, True])
def test_layouts_and_types(dt, view, split):
    run(2, 33, 5, 3, (16, 56, 56), dt=dt, split=split, view=view, norm=True, inverse=True)


@pytest.mark.parametrize("B,N,Hq,Hk", [(1, 1, 1, 1), (4, 1, 24, 24), (1, 17, 24, 1), (3, 16, 1, 0), (1, 300, 24, 24),
                                       (1, 2, 0, 3)])
def test_sizes(B, N, Hq, Hk):
    run(B, N, Hq, Hk, (16, 56, 56), norm=True, fractional=True)
    run(B, N, Hq, Hk, (16, 56, 56), batched=False)


def test_far_positions():
    """int32 positions up to 2^30: a binary32 angle would have no correct digit."""
    run(1, 64, 2, 2, (64, 64), dt="f32", top=1 << 30)


def test_positions_at_the_origin_are_the_identity():
    f = fqa()
    x = torch.randn(1, 2, 9, 128, device="cuda").bfloat16()
    pos = torch.zeros(9, 3, dtype=torch.int32, device="cuda")
    q, k = f.rotary(x, None, f.Rotary(pos, (16, 56, 56)))
    assert torch.equal(q, x) and k is None


def test_non_finite_values_stay_in_their_pair():
    f = fqa()
    x = torch.randn(1, 2, 9, 128, device="cuda")
    pos = torch.arange(9, dtype=torch.int32, device="cuda")[:, None]
    for split in (False, True):
        rot = f.Rotary(pos, (64,), split=split)
        want, _ = f.rotary(x, None, rot)
        y = x.clone()
        y[0, 0, 3, 5], y[0, 1, 4, 100] = float("nan"), float("inf")
        got, _ = f.rotary(y, None, rot)
        a, b = (5, 37) if split else (4, 5)
        bad = torch.zeros_like(x, dtype=torch.bool)
        bad[0, 0, 3, a] = bad[0, 0, 3, b] = True
        assert torch.isnan(got)[bad].all() and got[0, 1, 4, 100] == float("inf")
        bad[0, 1, 4, 100] = True
        assert torch.equal(got[~bad], want[~bad])


def test_inverse_returns_the_input():
    f = fqa()
    x = torch.randn(1, 3, 50, 128, device="cuda")
    rot = f.Rotary(torch.randint(0, 5000, (50, 2), dtype=torch.int32, device="cuda"), (64, 64))
    y, _ = f.rotary(x, None, rot)
    back, _ = f.rotary(y, None, rot, inverse=True)
    assert (back - x).abs().max() <= 2.0 ** -18 * x.abs().max()


def test_the_inverse_is_the_gradient():
    """d/dx of <g, rotary(x)> is the inverse rotation of g: against differences
    (the rotation is linear, so they are exact up to rounding)."""
    f = fqa()
    g = torch.randn(1, 1, 4, 128, device="cuda")
    rot = f.Rotary(torch.randint(0, 50, (4, 3), dtype=torch.int32, device="cuda"), (16, 56, 56))
    grad, _ = f.rotary(g, None, rot, inverse=True)
    x = torch.randn(1, 1, 4, 128, device="cuda")
    for c in (0, 1, 15, 16, 70, 127):
        e = torch.zeros_like(x)
        e[..., c] = 1.0
        diff = ((f.rotary(x + e, None, rot)[0] - f.rotary(x - e, None, rot)[0]) * g).sum(-1) / 2
        assert (diff - grad[..., c]).abs().max() <= 2.0 ** -16 * g.abs().sum(-1).max()


def test_in_place_and_empty():
    f = fqa()
    for split in (False, True):
        x, y = (torch.randn(2, 3, 30, 128, device="cuda").bfloat16() for _ in range(2))
        rot = f.Rotary(torch.randint(0, 500, (30, 2), dtype=torch.int32, device="cuda"), (64, 64), split=split)
        q, k = f.rotary(x, y, rot)
        f.rotary(x, y, rot, q_out=x, k_out=y)
        assert torch.equal(q, x) and torch.equal(k, y)
    rot = f.Rotary(torch.empty(0, 2, dtype=torch.int32, device="cuda"), (64, 64))
    q, _ = f.rotary(x[:, :, :0], None, rot)
    assert q.shape == (2, 3, 0, 128)


def test_attention_paths_take_positions():
    """fp8_attention(rot=...) is rotary() followed by the same call without it."""
    f = fqa()
    packed = torch.randn(1, 200, 3, 2, 128, device="cuda").bfloat16()
    q, k, v = (packed[:, :, i].transpose(1, 2) for i in range(3))
    v = v.contiguous()
    w = (1 + 0.1 * torch.randn(128, device="cuda")).bfloat16()
    rot = f.Rotary(torch.randint(0, 60, (200, 3), dtype=torch.int32, device="cuda"), (16, 56, 56), q_weight=w, k_weight=w)
    qr, kr = f.rotary(q, k, rot)
    s = f.softmax_scale()
    assert torch.equal(f.fp8_attention(q, k, v, s, rot=rot), f.fp8_attention(qr, kr, v, s))
    assert torch.equal(f.nvfp4_attention(q, k, v, s, rot=rot), f.nvfp4_attention(qr, kr, v, s))


def test_another_stream_and_a_replayed_graph():
    f = fqa()
    x = torch.randn(1, 4, 100, 128, device="cuda").bfloat16()
    rot = f.Rotary(torch.randint(0, 500, (100, 2), dtype=torch.int32, device="cuda"), (64, 64))
    want = f.rotary(x, x, rot)[1]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = f.rotary(x, x, rot, stream=side)[1]
    side.synchronize()
    assert torch.equal(want, got)
    xs = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = f.rotary(xs, None, rot)
    xs.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, y)


def test_refusals():
    f = fqa()
    q = torch.zeros(2, 3, 8, 128, device="cuda").bfloat16()
    pos = torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    rot = f.Rotary(pos, (128,))
    w = torch.ones(128, device="cuda")
    for bad in (lambda: f.rotary(q[..., :64], None, rot), lambda: f.rotary(q[0], None, rot),
                lambda: f.rotary(q.transpose(2, 3), None, rot), lambda: f.rotary(q, q[:, :, :4], rot),
                lambda: f.rotary(q, q.float(), rot), lambda: f.rotary(q, q[:1], rot), lambda: f.rotary(q.int(), None, rot),
                lambda: f.rotary(q, None, rot._replace(positions=pos[:7])),
                lambda: f.rotary(q, None, rot._replace(positions=pos.long())),
                lambda: f.rotary(q, None, rot._replace(positions=pos.expand(8, 2), axes=(64, 64))),
                lambda: f.rotary(q, None, rot._replace(positions=pos.expand(3, 8, 1))),
                lambda: f.rotary(q, None, rot._replace(axes=(130,))), lambda: f.rotary(q, None, rot._replace(theta=-1.0)),
                lambda: f.rotary(q, None, rot._replace(q_weight=w)), lambda: f.rotary(q, None, rot._replace(eps=-1.0)),
                lambda: f.rotary(q, None, rot, k_out=q), lambda: f.rotary(q, q, rot, q_out=q),
                lambda: f.rotary(q.transpose(0, 1)[:2], None, rot, q_out=q[:, :2]),
                lambda: f.rotary(q, q.clone(), rot, q_out=torch.empty_like(q).transpose(0, 1)),
                lambda: f.fp8_attention(q, q, q, 0.1, rot=rot._replace(positions=pos[:4]))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    out = torch.empty_like(q)
    with pytest.raises(ValueError, match="overlaps"):
        f.rotary(q, q.clone(), rot, q_out=out, k_out=out)


def test_rows_beyond_two_to_the_31_elements():
    f = fqa()
    N, H = 360_000, 48                        # 2.2e9 elements
    packed = torch.empty(1, N, H, 128, dtype=torch.bfloat16, device="cuda")
    packed[:, -50:].normal_()
    q = packed.transpose(1, 2)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[:, None]
    rot = f.Rotary(pos, (128,))
    y, _ = f.rotary(q, None, rot)
    want, _ = f.rotary(q[:, :, -50:], None, rot._replace(positions=pos[-50:].contiguous()))
    assert torch.equal(y[:, :, -50:], want)
