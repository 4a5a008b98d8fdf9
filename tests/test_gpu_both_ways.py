"""The native short cut of csrc/binding.cpp and the Python functions behind it take
and refuse the same calls, with the same results."""

import collections
import itertools

import numpy as np
import pytest
import torch

from tests import block_ref as R
from tests import test_gpu_microscale as rows
from tests import test_gpu_mx_matmul as product
from tests import test_gpu_rotary as rot

pytestmark = pytest.mark.gpu


@pytest.fixture
def checked(monkeypatch):
    import quantized_fp8_attention_b200 as f
    f.lib()
    monkeypatch.setattr(f, "_native", f._CheckedWay)
    return f


@pytest.mark.parametrize("test", [rows.test_refusals, rows.test_empty_rows, rows.test_norm_of_strided_and_broadcast_rows,
                                  rot.test_refusals, rot.test_in_place_and_empty, rot.test_attention_paths_take_positions,
                                  product.test_empty_sides, product.test_two_streams_at_once_and_replayed_graphs],
                         ids=lambda t: f"{t.__module__.split('.')[-1]}.{t.__name__}")
def test_the_checked_way_alone(checked, test):
    test()


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_formats_the_checked_way(checked, fmt):
    rows.test_special_rows(fmt)
    rows.test_strided_rows_and_leading_dimensions(fmt)
    rows.test_norm_of_zero_and_non_finite_rows(fmt)
    product.test_a_block_up_to_its_attention(fmt)
    for M, N, K in ((1, 1, 1), (17, 100, 160), (300, 1000, 480), (1500, 2048, 64)):
        product.check(M, N, K, fmt, M % 3, bias=True)


def outcome(call):
    """What a call gives: its tensors on the host, or the kind of its refusal."""
    def flat(v):
        if isinstance(v, torch.Tensor):
            return v.detach().cpu().view(torch.uint8).numpy().tobytes(), tuple(v.shape), v.dtype, tuple(v.stride())
        import quantized_fp8_attention_b200 as f
        if isinstance(v, f.Microscaled):       # scales of rows past M hold anything
            parts = R.held(v) if v.codes.shape[0] else [None if a is None else a.cpu() for a in v[:3]]
            return tuple(None if a is None else np.asarray(a).tobytes() for a in parts), v.cols, v.fmt
        return tuple(map(flat, v)) if isinstance(v, tuple) else v
    try:
        return flat(call())
    except Exception as e:
        return type(e)


def calls(f):
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.randn(30, 520, device="cuda", generator=g)
    xs = {}
    for name, t in (("bf16", wide.bfloat16()), ("f16", wide.half()), ("f32", wide)):
        xs[name] = t[:, :256]
        xs[name + " shifted"] = t[:, 3:259]
        xs[name + " 3d"] = t.view(5, 6, 520)[..., :256]
        xs[name + " rows"] = t[:, :256].contiguous().view(2, 15, 256)
    xs.update(one=wide[:1, :256].expand(30, 256), vector=wide[0, :256], turned=wide.T[:256], ints=wide[:, :256].int(),
              none=wide[:0, :256], empty=wide[:, :0], host=wide[:, :256].cpu(), f64=wide[:, :256].double(), number=3)
    for (name, x), fmt in itertools.product(xs.items(), (*R.FORMATS, "mxfp6", 1)):
        yield f"quantize {name} {fmt}", lambda x=x, fmt=fmt: f.mx_quantize(x, fmt)
    ws = (torch.ones(256, device="cuda"), torch.ones(256, device="cuda").bfloat16(), torch.ones(255, device="cuda"),
          torch.ones(512, device="cuda")[::2], torch.ones(256), None)
    for (name, x), (i, w), eps in itertools.product(xs.items(), enumerate(ws), (1e-6, 0, -1.0, float("nan"), "1")):
        yield f"norm {name} {i} {eps}", lambda x=x, w=w, eps=eps: f.mx_rms_norm(x, w, "mxfp8", eps=eps)
    for (name, x), (other, r) in itertools.product(xs.items(), xs.items()):
        yield f"norm {name} + {other}", lambda x=x, r=r: f.mx_rms_norm(x, ws[0], "nvfp4", residual=r)
    qs = {fmt: f.mx_quantize(xs["bf16"], fmt) for fmt in R.FORMATS}
    a = qs["nvfp4"]
    qs.update(narrow=f.mx_quantize(xs["bf16"][:, :224], "nvfp4"), codes=a._replace(codes=a.codes[:, :64]), plain=tuple(a),
              rows=a._replace(codes=a.codes[:20]), row=a._replace(row_scale=None), cols=a._replace(cols=255),
              cols0=a._replace(cols=0), colsf=a._replace(cols=256.0), fmt=a._replace(fmt="mxfp4"), half=a._replace(
                  row_scale=a.row_scale.half()), none=None)
    for (name, q), t in itertools.product(qs.items(), (0, 1, 2, 3, -1, True, "0", None)):
        yield f"back {name} {t}", lambda q=q, t=t: f.mx_dequantize(q, t)
    biases = (None, torch.ones(30, device="cuda"), torch.ones(31, device="cuda"), torch.ones(30, device="cuda").half())
    for (n1, p), (n2, q), (i, b) in itertools.product(qs.items(), qs.items(), enumerate(biases)):
        yield f"product {n1} {n2} {i}", lambda p=p, q=q, b=b: f.mx_matmul(p, q, bias=b, out_dtype=1)
    packed = torch.randn(2, 9, 5, 128, device="cuda", generator=g).bfloat16()
    q, k = packed[:, :, :3].transpose(1, 2), packed[:, :, 3:].transpose(1, 2)
    pos = torch.randint(0, 99, (9, 2), dtype=torch.int32, device="cuda", generator=g)
    base = f.Rotary(pos, (64, 64))
    rots = dict(base=base, lists=base._replace(axes=[64, 64]), odd=base._replace(axes=(63, 65)), wide=base._replace(axes=(64, 66)),
                floats=base._replace(axes=(64.0, 64.0)), split=base._replace(axes=(16, 24), split=True), one=base._replace(axes=(128,)),
                splitw=base._replace(axes=(16, 32), split=True), shared=base._replace(shared=True), flag=base._replace(split=1),
                theta=base._replace(theta=500), theta0=base._replace(theta=0), thetas=base._replace(theta="1"),
                batch=base._replace(positions=pos.expand(2, 9, 2).contiguous().float()), batch1=base._replace(positions=pos[None]),
                batch3=base._replace(positions=pos.expand(3, 9, 2).contiguous()), long=base._replace(positions=pos.long()),
                short=base._replace(positions=pos[:8]), apart=base._replace(positions=pos.T.contiguous().T),
                weight=base._replace(q_weight=torch.ones(128, device="cuda").bfloat16()), other=base._replace(
                    k_weight=torch.ones(128, device="cuda")), eps=base._replace(eps=-1.0), eps0=base._replace(eps=0),
                plain=tuple(base), none=None)
    inputs = dict(views=(q, k), alone=(q, None), tokens=(q, k[:, :, :8]), types=(q, k.float()), batch=(q, k[:1]),
                  three=(q[0], None), narrow=(q[..., :64], None), turned=(q.transpose(2, 3), None), host=(q.cpu(), None),
                  hosts=(q, k.cpu()), noheads=(q[:, :0], k), empty=(q[:, :, :0], None))
    for (n1, r), (n2, (a1, a2)), inverse in itertools.product(rots.items(), inputs.items(), (False, True, 1)):
        yield f"rotary {n1} {n2} {inverse}", lambda r=r, a1=a1, a2=a2, inverse=inverse: f.rotary(a1, a2, r, inverse=inverse)


def test_the_same_calls_are_taken_and_refused(monkeypatch):
    import quantized_fp8_attention_b200 as f
    f.lib()
    native = f._native
    assert native is not f._CheckedWay, "the binding is built for this torch"
    taken = collections.Counter()
    for name, call in calls(f):
        monkeypatch.setattr(f, "_native", native)
        short = outcome(call)
        monkeypatch.setattr(f, "_native", f._CheckedWay)
        assert outcome(call) == short, name
        taken[name.split()[0]] += not isinstance(short, type)
    # of each kind at least the right ones: 14 inputs x 3 formats; 14 with a weight
    # of FP32 and 4 of BF16, with two eps, and 40 pairs with a residual; 5 operands
    # x 4 types; 5 pairs x 2 biases; 10 rotations x 3 inputs x 3 directions
    for kind, least in (("quantize", 42), ("norm", 76), ("back", 20), ("product", 10), ("rotary", 90)):
        assert taken[kind] >= least, (kind, taken[kind])
    assert f.fqa_debug_status()[0] == f.FQA_OK
