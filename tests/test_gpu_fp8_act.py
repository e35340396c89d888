"""Activations with their checkpoint in 8 bits, against the 64-bit formulas of fp8_ref.py.

What is quantised from a computed value: the kernel's fp32 value v' is within d = 16 x 2^-24 (|x| s, the product
before the activation's factor) of v; its block's scale is within that of the largest value's, so a stored value
may be the neighbour of the definition's where v r lies within d of a border. Allowed is therefore half a step of the
format more than its own rounding: |value - v| <= step(v) / 2 + d, step the distance of two codes around v r. Saved codes
are exact and compared byte for byte, and so is everything of ReLU, whose values are the inputs or zero.
"""
import numpy as np
import pytest
import torch

import fp8_ref as R
import gemm_epilogue_persistent_amd as gep
from test_gpu_fp8 import SENTINEL, TYPES, announce, check_quantized, dirty, operand, stored, values

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "relu_sq", "gelu_tanh", "silu"]
SIZES = [(1, 1), (1, 520), (3, 16), (65, 200), (130, 1000), (257, 136), (128, 128), (300, 135)]


def ordinary(seed, rows, cols, kind):
    """Values of a model's size, some far out in the activations' tails, a zero row and a zero column."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * 3
    far = torch.rand(rows, cols, generator=g) < 0.02
    x = torch.where(far, x * 20, x)
    if rows > 4:
        x[3] = 0
        x[:, cols // 2] = 0
    return x.to(TYPES[kind])


def check_values(q, v, off):
    """q holds the nearest values of the format to v (rows, k), or to anything within `off` of it."""
    codes, scales = q.codes.cpu().numpy(), R.load_scales(q.scales.cpu().numpy(), v.shape[0])
    rows, k = v.shape
    nb = -(-k // 128)
    assert (codes[:, k:] == 0).all() and (scales[:, nb:] == 0).all() and np.isfinite(scales).all()
    got = R.values(codes, scales[:, :nb], k)
    pad = lambda t: np.pad(t, ((0, 0), (0, nb * 128 - k))).reshape(rows, nb, 128)  # noqa: E731
    top, slack = pad(np.abs(v)).max(-1), pad(off).max(-1)
    # the scale is the definition's of a largest magnitude within `off`
    lo, hi = 1 / R.factor(np.maximum(top - slack, 0)), 1 / R.factor(top + slack)
    s = scales[:, :nb].astype(np.float64)
    assert (s >= lo * (1 - 2.0 ** -24)).all() and (s <= hi * (1 + 2.0 ** -24)).all()
    spread = R.spread(s, rows, k, False)
    u = np.abs(v) / spread
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(u, 2.0 ** -20))), -6) - 3) * spread
    err = np.abs(got - v)
    # (a value just below a power of two may be rounded as one above it: twice the step only for what `off` moves)
    tol = step / 2 * (1 + 2.0 ** -22) + off + 2.0 ** -22 * np.abs(v)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} out, worst {np.max(err / tol):.4g}"


def evaluation(x, v, act):
    """How far the kernel's fp32 value of act(x) (or its slope) may be off."""
    return 16 * 2.0 ** -24 * np.abs(v) + (2.0 ** -22 * np.minimum(1, np.abs(x)) if act in ("gelu_tanh", "silu") else 0)


def check_plain(t, v, off, kind):
    eps = torch.finfo(TYPES[kind]).eps / 2
    g = t.double().cpu().numpy()
    tol = off * (1 + eps) + eps * np.abs(v) + torch.finfo(TYPES[kind]).tiny
    assert (np.abs(g - v) <= tol).all(), f"worst {np.max(np.abs(g - v) / tol):.4g}"


def framed(rows, cols, kind):
    buf = torch.full((rows + 1, cols + 11), SENTINEL, dtype=TYPES[kind], device="cuda")
    return buf[:rows, 3:3 + cols], buf


def frame_kept(buf, rows, cols):
    return bool((buf[rows:] == SENTINEL).all()) and bool((buf[:, :3] == SENTINEL).all()) and bool((buf[:, 3 + cols:] == SENTINEL).all())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols, act, kind):
    announce(f"fp8 act {rows}x{cols} {act} {kind}")
    x = ordinary(rows + cols, rows, cols, kind)
    x64 = x.double().numpy()
    y64 = R.act(x64, act)
    view, buf = framed(rows, cols, kind)
    view.copy_(x)
    saved, q = dirty(rows, cols), dirty(rows, cols)
    y, ybuf = framed(rows, cols, kind)
    assert gep.fp8_act(view, act, saved=saved, q=q, y=y) is y
    check_quantized(saved, x64)
    off = evaluation(x64, y64, act)
    if act in ("none", "relu") and kind != "f32":
        check_quantized(q, y64)
    else:
        check_values(q, y64, off)
    if kind != "f16" or act != "relu_sq":  # (squares that pass f16's largest value)
        check_plain(y, y64, off, kind)
    assert frame_kept(ybuf, rows, cols) and frame_kept(buf, rows, cols) and torch.equal(view.cpu(), x)
    # each output alone, and y in the place of x
    for kw in (dict(saved=dirty(rows, cols)), dict(q=dirty(rows, cols))):
        t = gep.fp8_act(view, act, **kw)
        assert torch.equal(t.codes, (saved if "saved" in kw else q).codes)
    assert torch.equal(gep.fp8_act(view, act), y)
    gep.fp8_act(view, act, y=view)
    assert torch.equal(view, y)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(rows, cols, act, kind):
    announce(f"fp8 act backward {rows}x{cols} {act} {kind}")
    x = ordinary(rows + 2 * cols, rows, cols, "f32").double().numpy()
    codes, scales = R.quantize(x)
    kept = stored(codes, scales, cols)
    xh = R.values(codes, scales, cols).astype(np.float32).astype(np.float64)
    dy = torch.randn(rows, cols, generator=torch.Generator().manual_seed(1)).to(TYPES[kind])
    dy64 = dy.double().numpy()
    want, y64 = dy64 * R.slope(xh, act), R.act(xh, act)
    view, vbuf = framed(rows, cols, kind)
    view.copy_(dy)
    dx, dbuf = framed(rows, cols, kind)
    y, ybuf = framed(rows, cols, kind)
    q, qt, yt = dirty(rows, cols), dirty(cols, rows), dirty(cols, rows)
    gep.fp8_act_backward(view, kept, act, dx=dx, q=q, qt=qt, y=y, yt=yt)
    # the slope's own error scales with |dy|; |slope| reaches 1.13, and 2 |x| for ReLU^2
    off = np.abs(dy64) * evaluation(np.ones_like(xh), R.slope(xh, act), act) + 2.0 ** -23 * np.abs(want)
    offy = evaluation(xh, y64, act) + 2.0 ** -23 * np.abs(y64)
    exact = act in ("none", "relu") and kind != "f32"
    if exact:
        check_quantized(q, want)
        check_quantized(qt, want.T)
    else:
        check_values(q, want, off)
        check_values(qt, want.T, off.T)
    check_values(yt, y64.T, offy.T)
    check_plain(dx, want, off, kind)
    if kind != "f16" or act != "relu_sq":
        check_plain(y, y64, offy, kind)
    for b in (vbuf, dbuf, ybuf):
        assert frame_kept(b, rows, cols)
    # each output alone
    for name, t in (("q", q), ("qt", qt), ("yt", yt)):
        alone = dirty(*t.shape)
        gep.fp8_act_backward(None if name == "yt" else view, kept, act, **{name: alone})
        assert torch.equal(alone.codes, t.codes)
    z = torch.empty(rows, cols, dtype=TYPES[kind], device="cuda")
    gep.fp8_act_backward(None, kept, act, y=z)
    assert torch.equal(z, y)
    gep.fp8_act_backward(view, kept, act, dx=view)
    assert torch.equal(view, dx)


@pytest.mark.parametrize("act", ["relu_sq", "gelu_tanh", "silu"])
def test_slope_is_the_difference(act):
    """dx against central differences of the forward formula."""
    announce(f"fp8 act differences {act}")
    x = np.linspace(-7, 7, 128 * 9).reshape(9, 128)
    codes, scales = R.quantize(x)
    xh = R.values(codes, scales, 128).astype(np.float32).astype(np.float64)
    dx = torch.empty(9, 128, device="cuda")
    gep.fp8_act_backward(torch.ones(9, 128, device="cuda"), stored(codes, scales, 128), act, dx=dx)
    h = 1e-4  # (third derivatives below 10: an error below 2e-8, and 1e-12 of cancellation)
    diff = (R.act(xh + h, act) - R.act(xh - h, act)) / (2 * h)
    diff = np.where(xh == 0, R.slope(xh, act), diff) if act == "relu_sq" else diff
    assert np.abs(dx.double().cpu().numpy() - diff).max() < 1e-7 + 2.0 ** -19 * np.abs(diff).max()


def test_far_values():
    """Slopes and values at the ends of fp32's range are finite and the limits."""
    announce("fp8 act far values")
    x = torch.tensor([3e38, -3e38, 1e20, -1e20, 100.0, -100.0, 1e-38, 0.0]).repeat_interleave(128).view(8, 128)
    kept = gep.fp8_quantize(x.cuda())
    for act, up in (("relu", 1), ("gelu_tanh", 1), ("silu", 1)):
        dx, y = torch.empty(8, 128, device="cuda"), torch.empty(8, 128, device="cuda")
        gep.fp8_act_backward(torch.ones(8, 128, device="cuda"), kept, act, dx=dx, y=y)
        xh = gep.fp8_dequantize(kept, dtype=torch.float32)
        assert torch.equal(dx[0::2][:3], torch.full((3, 128), float(up), device="cuda"))
        assert (dx[1:6:2].abs() < 1e-30).all()
        assert torch.equal(y[0::2][:3], xh[0::2][:3]) and (y[1:6:2].abs() < 1e-30).all()


def test_not_finite():
    """A NaN in x makes its block of the checkpoint NaN, and with it that block's gradients."""
    announce("fp8 act not finite")
    x = ordinary(3, 200, 300, "bf16")
    x[17, 140] = float("nan")
    kept, q = dirty(200, 300), dirty(200, 300)
    gep.fp8_act(x.cuda(), "silu", saved=kept, q=q)
    assert torch.equal(gep.fp8_dequantize(kept).isnan().nonzero(), gep.fp8_dequantize(q).isnan().nonzero())
    dx, qt = torch.empty(200, 300, device="cuda", dtype=torch.bfloat16), dirty(300, 200)
    gep.fp8_act_backward(torch.ones_like(dx), kept, "silu", dx=dx, qt=qt)
    bad = torch.zeros(200, 300, dtype=torch.bool, device="cuda")
    bad[17, 128:256] = True
    assert torch.equal(dx.isnan(), bad)
    t = torch.zeros(300, 200, dtype=torch.bool, device="cuda")
    t[128:256, :128] = True
    assert torch.equal(gep.fp8_dequantize(qt).isnan(), t)


def test_transposed_checkpoint():
    """act none: the checkpoint's blocks along the other axis, the rounding of its values."""
    announce("fp8 act transposed checkpoint")
    codes, scales = operand(3, 270, 400)
    kept, yt = stored(codes, scales, 400), dirty(400, 270)
    gep.fp8_act_backward(None, kept, "none", yt=yt)
    v = R.values(codes, scales, 400)
    check_values(yt, v.T, 2.0 ** -24 * np.abs(v.T))


def test_refusals():
    x = torch.zeros(16, 64, device="cuda")
    k = gep.fp8_empty(16, 64)
    for kw in (dict(saved=gep.fp8_empty(16, 64, tiles=True)), dict(q=gep.fp8_empty(16, 80)), dict(y=torch.zeros(16, 63, device="cuda")),
               dict(saved=k, q=k), dict(saved=gep.fp8_empty(16, 64, groups=2))):
        with pytest.raises(ValueError):
            gep.fp8_act(x, "silu", **kw)
    with pytest.raises(ValueError):
        gep.fp8_act(x, "tanh", saved=k)
    with pytest.raises(TypeError):
        gep.fp8_act(x, "silu", y=x.bfloat16())
    with pytest.raises(TypeError):
        gep.fp8_act(x, "silu", saved=x)
    with pytest.raises(gep.GemmError):
        gep.fp8_act(x.as_strided((2, 8), (8, 1)), "silu", y=x.as_strided((2, 8), (64, 1)))
    for args, kw in (((x, k, "silu"), {}), ((None, k, "silu"), {}), ((None, k, "silu"), dict(dx=x)), ((x, k, "silu"), dict(yt=gep.fp8_empty(64, 16))),
                     ((x, k, "silu"), dict(qt=gep.fp8_empty(16, 64))), ((x, k, "tanh"), dict(dx=x)),
                     ((x, gep.fp8_empty(16, 64, tiles=True), "silu"), dict(dx=x))):
        with pytest.raises(ValueError):
            gep.fp8_act_backward(*args, **kw)
    with pytest.raises(TypeError):
        gep.fp8_act_backward(x, x, "silu", dx=x)
    with pytest.raises(TypeError):
        gep.fp8_act_backward(x, k, "silu", dx=x, y=x.bfloat16())
    with pytest.raises(gep.GemmError):
        gep.fp8_act_backward(x, k, "silu", q=k)
    s, t = gep.fp8_empty(64, 64), gep.fp8_empty(64, 64)
    with pytest.raises(gep.GemmError):
        gep.fp8_act_backward(torch.zeros(64, 64, device="cuda"), s, "silu", q=t, qt=t)
    with pytest.raises(gep.GemmError):
        gep.fp8_act_backward(x, k, "silu", dx=x, y=x)
