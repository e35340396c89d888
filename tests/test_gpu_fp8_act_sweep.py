"""Seeded random sweep of the activations with their checkpoint in 8 bits and of their backward pass: sizes, types, activations, strides,
odd starts, subsets of the outputs and results in the place of their inputs drawn together, each case against the 64-bit
formulas. GEP_SWEEP_CASES sets the number of cases of each kind (default 60; case i draws from seed 100 + i).

Tolerances of the smooth activations, in half steps h = 2^-24 of the value x s, s = 1 / (1 + e^-z): z is off by 7 roundings of itself and
its product with log2 e by 2 more, so that e^-z is off by 9 |z| h of itself, s by 9 |z| (1 - s) h and 1 - s by 9 |z| s h; the exponential and
the reciprocal 2 each, sums and products 1 each: at most 16 h. The slope is s (1 + x (1 - s) z'), each factor off by its own. Where e^-z
leaves fp32 (z below -83) results are 0 or nearly: 2^-108, e^-75, covers both.
"""
import os
import random

import numpy as np
import pytest
import torch

import fp8_ref as R
import gemm_epilogue_persistent_amd as gep
from test_gpu_fp8 import SENTINEL, TYPES, announce, check_quantized, dirty, stored
from test_gpu_fp8_act import ACTS, check_plain, check_values, ordinary
from test_gpu_fp8_sweep import spread

pytestmark = pytest.mark.gpu

CASES = int(os.environ.get("GEP_SWEEP_CASES", "60"))
H = 2.0 ** -24
FLOOR = 2.0 ** -108


def inner(x, act):
    """z and dz / dx of x / (1 + e^-z)."""
    if act == "silu":
        return x, np.ones_like(x)
    c = 2 * np.sqrt(2 / np.pi)
    return c * (x + 0.044715 * x ** 3), c * (1 + 3 * 0.044715 * x * x)


def value_error(x, act):
    v = np.abs(R.act(x, act))
    if act not in ("gelu_tanh", "silu"):
        return 2 * H * v
    z = inner(x, act)[0]
    with np.errstate(over="ignore"):
        rest = 1 / (1 + np.exp(z))
    return (9 * np.abs(z) * rest + 16) * H * v + FLOOR


def slope_error(x, act):
    if act not in ("gelu_tanh", "silu"):
        return 2 * H * np.abs(R.slope(x, act))
    z, dz = inner(x, act)
    with np.errstate(over="ignore"):
        s, rest = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    part, steps = np.abs(x) * rest * dz, 9 * np.abs(z)
    return H * s * ((steps * rest + 16) * (1 + part) + steps * s * part) + FLOOR


class Place:
    """A matrix (rows, cols) with a row stride and a start of its own amid sentinels."""

    def __init__(self, r, rows, cols, kind, value=None):
        self.pad, self.at = r.randint(0, 9), r.randint(0, 5)
        self.buf = torch.full((rows * (cols + self.pad) + self.at + 1,), SENTINEL, dtype=TYPES[kind], device="cuda")
        self.view = self.buf[self.at:self.at + rows * (cols + self.pad)].view(rows, cols + self.pad)[:, :cols]
        if value is not None:
            self.view.copy_(value)

    def frame_kept(self):
        kept = self.view.clone()
        self.view.fill_(SENTINEL)
        ok = bool((self.buf == SENTINEL).all())
        self.view.copy_(kept)
        return ok


def subset(r, names):
    some = [n for n in names if r.random() < 0.6]
    return some or [r.choice(names)]


@pytest.mark.parametrize("i", range(CASES))
def test_forward(i):
    r = random.Random(100 + i)
    rows, cols, kind, act = spread(r, 1, 900), spread(r, 1, 1500), r.choice(list(TYPES)), r.choice(ACTS)
    some, place = subset(r, ["saved", "q", "y"]), r.random() < 0.3
    announce(f"fp8 act sweep {i}: {rows}x{cols} {kind} {act} {some} in place {place}")
    x = ordinary(1000 + i, rows, cols, kind)
    if kind == "f16" and act == "relu_sq":
        x = x.clamp(-200, 200)  # (squares within F16's range)
    x64 = x.double().numpy()
    y64 = R.act(x64, act)
    src = Place(r, rows, cols, kind, x)
    y = None if "y" not in some else (src if place else Place(r, rows, cols, kind))
    saved, q = (dirty(rows, cols) if n in some else None for n in ("saved", "q"))
    gep.fp8_act(src.view, act, saved=saved, q=q, y=y.view if y else None)
    if saved is not None:
        check_quantized(saved, x64)
    if q is not None:
        if act in ("none", "relu") and kind != "f32":  # (q's values are x's own or 0, whose products with r are exact)
            check_quantized(q, y64)
        else:
            check_values(q, y64, value_error(x64, act))
    if y is not None:
        check_plain(y.view, y64, value_error(x64, act), kind)
        assert y.frame_kept()
    assert src.frame_kept() and (y is src or torch.equal(src.view.cpu(), x))


@pytest.mark.parametrize("i", range(CASES))
def test_backward(i):
    r = random.Random(100 + i)
    rows, cols, kind, act = spread(r, 1, 900), spread(r, 1, 1500), r.choice(list(TYPES)), r.choice(ACTS)
    some, place = subset(r, ["dx", "q", "qt", "y", "yt"]), r.random() < 0.3
    announce(f"fp8 act backward sweep {i}: {rows}x{cols} {kind} {act} {some} in place {place}")
    x = ordinary(1000 + i, rows, cols, "f32").double().numpy()
    if kind == "f16" and act == "relu_sq":
        x = np.clip(x, -200, 200)
    codes, scales = R.quantize(x)
    kept = stored(codes, scales, cols)
    xh = R.values(codes, scales, cols).astype(np.float32).astype(np.float64)
    dy = torch.randn(rows, cols, generator=torch.Generator().manual_seed(i)).to(TYPES[kind])
    grad = any(n in some for n in ("dx", "q", "qt"))
    dy64 = dy.double().numpy()
    want, y64 = dy64 * R.slope(xh, act), R.act(xh, act)
    off = np.abs(dy64) * slope_error(xh, act) + 2 * H * np.abs(want)
    offy = value_error(xh, act) + 2 * H * np.abs(y64)
    src = Place(r, rows, cols, kind, dy) if grad else None
    dx = None if "dx" not in some else (src if place else Place(r, rows, cols, kind))
    y = Place(r, rows, cols, kind) if "y" in some else None
    m = {n: dirty(*((rows, cols) if n == "q" else (cols, rows))) for n in ("q", "qt", "yt") if n in some}
    gep.fp8_act_backward(src.view if grad else None, kept, act, dx=dx.view if dx else None, y=y.view if y else None, **m)
    if "q" in m:
        check_values(m["q"], want, off)
    if "qt" in m:
        check_values(m["qt"], want.T, off.T)
    if "yt" in m:
        check_values(m["yt"], y64.T, offy.T)
    if dx is not None:
        check_plain(dx.view, want, off, kind)
    if y is not None:
        check_plain(y.view, y64, offy, kind)
    for p in (src, dx, y):
        assert p is None or p.frame_kept()
    assert src is None or dx is src or torch.equal(src.view.cpu(), dy)


@pytest.mark.parametrize("act,kind", [("gelu_tanh", "f32"), ("silu", "f32"), ("gelu_tanh", "bf16"), ("silu", "f16")])
def test_negative_tail(act, kind):
    """Values and slopes far down the negative tail, relative to themselves: every block holds values of one size, so that a
    checkpoint and q keep their digits."""
    announce(f"fp8 act tail {act} {kind}")
    end = 9.5 if act == "gelu_tanh" else 79.0
    top = np.linspace(0.5, end if kind != "f16" else 9.0, 300)  # (F16 ends at 2^-24)
    x = torch.from_numpy(-top[:, None] * (1 - np.arange(128)[None, :] / 512)).to(TYPES[kind])
    x64 = x.double().numpy()
    saved, q, y = dirty(300, 128), dirty(300, 128), torch.empty_like(x, device="cuda")
    gep.fp8_act(x.cuda(), act, saved=saved, q=q, y=y)
    check_quantized(saved, x64)
    check_values(q, R.act(x64, act), value_error(x64, act))
    check_plain(y, R.act(x64, act), value_error(x64, act), kind)
    codes, scales = R.quantize(x64)
    xh = R.values(codes, scales, 128).astype(np.float32).astype(np.float64)
    dx, qd, yt = torch.empty(300, 128, device="cuda"), dirty(300, 128), dirty(128, 300)
    gep.fp8_act_backward(torch.ones(300, 128, device="cuda"), saved, act, dx=dx, q=qd, yt=yt)
    check_plain(dx, R.slope(xh, act), slope_error(xh, act), "f32")
    check_values(qd, R.slope(xh, act), slope_error(xh, act))
    check_values(yt, R.act(xh, act).T, value_error(xh, act).T)
