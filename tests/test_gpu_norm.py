"""RMS norm with residual and MX output, and its gradients, against 64-bit formulas.

Tolerances. h is the rounded sum and is compared exactly. With u = 2^-24 (fp32's half step) a sum
of n squares differs by at most (n + 2) u of itself, whatever its order; rstd's relative error is
half of that plus 4 u (mean, eps, root, quotient), y's two products add 2 u, the output type half a
step. The MX output may be the rounding of any value that close to y.
"""
import sys

import numpy as np
import pytest
import torch

import gemm_epilogue_persistent_amd as gep
import mx_ref as R

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24
SENTINEL = 77.0


def announce(name):
    print(f"[case] {name}", flush=True)
    sys.stdout.flush()


def data(seed, rows, cols, kind, n):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(rows, cols, generator=g).to(TYPES[kind]) for _ in range(n)] + [
        (1 + 0.3 * torch.randn(cols, generator=g)).to(TYPES[kind])]


def padded(t):
    """The matrix inside a wider buffer, at an odd column."""
    buf = torch.full((t.shape[0], t.shape[1] + 5), SENTINEL, dtype=t.dtype, device="cuda")
    v = buf[:, 3:3 + t.shape[1]]
    v.copy_(t)
    return v, buf


def unharmed(buf, cols):
    return bool((buf[:, :3] == SENTINEL).all()) and bool((buf[:, 3 + cols:] == SENTINEL).all())


def check_close(got, want, rel, kind, name):
    eps = torch.finfo(TYPES[kind]).eps / 2 if kind else 0.0
    g = got.double().cpu().numpy()
    tol = np.abs(want) * (rel + eps + rel * eps) + (torch.finfo(TYPES[kind]).tiny if kind else 0)
    err = np.abs(g - want)
    assert np.isfinite(g).all(), name
    assert (err <= tol).all(), f"{name}: {(err > tol).sum()} out, worst {np.max(err / np.maximum(tol, 1e-300)):.3g}"


def check_mx(q, y, rel, fmt):
    """Each value is the rounding of y (1 + d), |d| <= rel, under the scale of such a block."""
    k = y.shape[1]
    v = R.values(R.unpack(q.codes.cpu().numpy(), fmt), R.load_scales(q.scales.cpu().numpy(), y.shape[0])[:, : -(-k // 32)], fmt, k)
    lo, hi = np.full(y.shape, np.inf), np.zeros(y.shape)
    for f in (1 - rel, 1 + rel):
        s = R.scale_bytes(y * f, fmt)
        for f2 in (1 - rel, 1 + rel):
            c = R.round_code(np.abs(R.blocks(y * f2)) / 2.0 ** (s[..., None] - 127.0), fmt)
            a = R.values(c.reshape(y.shape[0], -1), s, fmt, k)
            lo, hi = np.minimum(lo, a), np.maximum(hi, a)
    assert (np.abs(v) >= lo).all() and (np.abs(v) <= hi).all()
    assert (np.sign(v) * np.sign(y) >= 0).all()


SHAPES = [(1, 1), (1, 4096), (3, 64), (5, 500), (1030, 72), (1030, 1000), (1025, 2001), (1024, 4096), (7, 2048), (4, 4100),
          (9, 8192), (3, 10000), (2, 32768), (2, 40001)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, kind):
    announce(f"rmsnorm {rows}x{cols} {kind}")
    x, r, w = data(rows + cols, rows, cols, kind, 2)
    eps = 1e-5
    rel_r = (cols + 2) * U / 2 + 4 * U
    rel = rel_r + 2 * U
    (xd, xb), (rd, rb), wd = padded(x), padded(r), w.cuda()
    h, hb = padded(torch.zeros_like(x))
    y, yb = padded(torch.zeros_like(x))
    rstd = torch.full((rows,), SENTINEL, device="cuda")
    for residual in (True, False):
        want_h = (x.float() + r.float()).to(x.dtype) if residual else x
        h64 = want_h.double().numpy()
        want_r = 1 / np.sqrt((h64 ** 2).mean(1) + eps)
        want_y = h64 * want_r[:, None] * w.double().numpy()
        for fmt in ("e4m3", "e2m1"):
            q = gep.mx_empty(rows, cols, fmt)
            q.codes.fill_(0x33)
            q.scales.fill_(0xFF)
            gep.rmsnorm(xd, wd, residual=rd if residual else None, eps=eps, h=h if residual else None,
                        y=y if fmt == "e4m3" else None, q=q, rstd=rstd)
            check_mx(q, want_y, rel, fmt)
            nb = -(-cols // 32)
            assert (R.load_scales(q.scales.cpu().numpy(), rows)[:, nb:] == 0).all()
        if residual:
            assert torch.equal(h.cpu(), want_h)
        check_close(rstd, want_r, rel_r, "f32", "rstd")
        check_close(y, want_y, rel, kind, "y")
        assert unharmed(hb, cols) and unharmed(yb, cols) and unharmed(xb, cols)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(3, 64), (1100, 4096), (5, 6000), (2, 40001)])
def test_forward_in_place(rows, cols, kind):
    """h in the place of x or of the residual; y alone, allocated."""
    announce(f"rmsnorm in place {rows}x{cols} {kind}")
    x, r, w = data(7, rows, cols, kind, 2)
    h = torch.empty(rows, cols, dtype=x.dtype, device="cuda")
    y = gep.rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), h=h)
    for first in (True, False):
        a, b = x.cuda(), r.cuda()
        got = gep.rmsnorm(a, w.cuda(), residual=b, h=a if first else b)
        assert torch.equal(got, y) and torch.equal(a if first else b, h)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols, kind):
    """dx: each of its terms carries y's error; the mean of p n another (cols + 4) u of sum |p n| / cols;
    the sum is rounded once. dw: (rows + 6) u of sum |dy n|."""
    announce(f"rmsnorm backward {rows}x{cols} {kind}")
    dy, h, dres, w = data(rows + cols, rows, cols, kind, 3)
    h64, dy64, w64 = h.double().numpy(), dy.double().numpy(), w.double().numpy()
    rstd = torch.from_numpy(1 / np.sqrt((h64 ** 2).mean(1) + 1e-5)).float()
    r64 = rstd.double().numpy()[:, None]
    n, p = h64 * r64, dy64 * w64
    mean = (p * n).mean(1, keepdims=True)
    mean_err = (cols + 6) * U * np.abs(p * n).mean(1, keepdims=True)
    eps = torch.finfo(TYPES[kind]).eps / 2
    (dyd, _), (hd, _), (dresd, _), wd = padded(dy), padded(h), padded(dres), w.cuda()
    for res in (True, False):
        want = r64 * (p - n * mean) + (dres.double().numpy() if res else 0)
        mag = r64 * (np.abs(p) + np.abs(n * mean)) + (np.abs(dres.double().numpy()) if res else 0)
        dx, dxb = padded(torch.zeros_like(h))
        dw = torch.full((cols,), SENTINEL, device="cuda")
        gep.rmsnorm_backward(dyd, hd, wd, rstd.cuda(), dx=dx, dw=dw, dres=dresd if res else None)
        err = np.abs(dx.double().cpu().numpy() - want)
        tol = (8 * U * mag + r64 * np.abs(n) * mean_err) * (1 + eps) + eps * np.abs(want) + torch.finfo(TYPES[kind]).tiny
        assert (err <= tol).all(), f"dx worst {np.max(err / tol):.3g}"
        assert unharmed(dxb, cols)
        err = np.abs(dw.double().cpu().numpy() - (dy64 * n).sum(0))
        tol = (rows + 6) * U * np.abs(dy64 * n).sum(0) + 1e-38
        assert (err <= tol).all(), f"dw worst {np.max(err / tol):.3g}"


def test_backward_against_differences():
    """The gradients against central differences of the 64-bit forward pass."""
    announce("rmsnorm backward against differences")
    rows, cols, eps, step = 3, 70, 1e-5, 1e-5
    dy, h, w = data(3, rows, cols, "f32", 2)
    h64, dy64, w64 = h.double().numpy(), dy.double().numpy(), w.double().numpy()

    def loss(hh, ww):
        return (dy64 * hh / np.sqrt((hh ** 2).mean(1, keepdims=True) + eps) * ww).sum()

    rstd = torch.from_numpy(1 / np.sqrt((h64 ** 2).mean(1) + eps)).float().cuda()
    dx, dw = gep.rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd)
    for i, j in ((0, 0), (1, 33), (2, 69)):
        a, b = h64.copy(), h64.copy()
        a[i, j] += step
        b[i, j] -= step
        diff = (loss(a, w64) - loss(b, w64)) / (2 * step)
        # (differences: step^2 of the third derivative, 2^-53 / step of the loss; the kernel: 2^-24 x 100)
        assert abs(dx[i, j].item() - diff) <= 1e-5 * (1 + abs(diff))
    for j in (0, 40, 69):
        a, b = w64.copy(), w64.copy()
        a[j] += step
        b[j] -= step
        diff = (loss(h64, a) - loss(h64, b)) / (2 * step)
        assert abs(dw[j].item() - diff) <= 1e-5 * (1 + abs(diff))


@pytest.mark.parametrize("rows,cols", [(40, 256), (700, 3000), (3, 40001)])
def test_backward_in_place_and_repeatable(rows, cols):
    announce(f"rmsnorm backward in place {rows}x{cols}")
    dy, h, dres, w = data(11, rows, cols, "bf16", 3)
    rstd = torch.rand(rows, device="cuda") + 0.5
    args = (h.cuda(), w.cuda(), rstd)
    ws = torch.full((gep.rmsnorm_backward_workspace(rows, cols),), 255, dtype=torch.uint8, device="cuda")
    dx, dw = gep.rmsnorm_backward(dy.cuda(), *args, dres=dres.cuda(), workspace=ws)
    for first in (True, False):
        a, b = dy.cuda(), dres.cuda()
        dx2, dw2 = gep.rmsnorm_backward(a, *args, dres=b, dx=a if first else b, workspace=ws)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_backward_no_rows():
    announce("rmsnorm backward without rows")
    z = torch.empty(0, 100, device="cuda")
    dw = torch.full((100,), SENTINEL, device="cuda")
    dx, _ = gep.rmsnorm_backward(z, z, torch.ones(100, device="cuda"), torch.empty(0, device="cuda"), dw=dw)
    assert dx.shape == (0, 100) and (dw == 0).all()


def test_zero_and_huge_rows():
    """A row of zeros gives zeros (rstd = eps^(-1/2)); a NaN stays in its row."""
    announce("rmsnorm zero rows and NaN")
    x = torch.randn(4, 300, device="cuda")
    x[1] = 0
    x[2, 7] = float("nan")
    rstd = torch.empty(4, device="cuda")
    q = gep.mx_empty(4, 300, "e4m3")
    y = torch.empty_like(x)
    gep.rmsnorm(x, torch.ones(300, device="cuda"), eps=1e-6, y=y, q=q, rstd=rstd)
    assert (y[1] == 0).all() and abs(rstd[1].item() - 1000) < 1e-3
    assert y[2].isnan().all() and not y[[0, 1, 3]].isnan().any()
    v = gep.mx_dequantize(q)
    assert v[2].isnan().all() and not v[[0, 1, 3]].isnan().any()


def test_python_refusals():
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    rstd = torch.ones(4, device="cuda")
    for kw in (dict(h=x), dict(q=gep.mx_empty(4, 32, "e4m3")), dict(residual=x[:2]), dict(y=x.t()), dict(rstd=rstd[:3]),
               dict(rstd=rstd.double())):
        with pytest.raises(ValueError):
            gep.rmsnorm(x, w, **kw)
    for kw in (dict(residual=x.half()), dict(y=x.half())):
        with pytest.raises(TypeError):
            gep.rmsnorm(x, w, **kw)
    with pytest.raises(ValueError):
        gep.rmsnorm(x, w[:32])
    with pytest.raises(ValueError):
        gep.rmsnorm(x, w.half())
    with pytest.raises(gep.GemmError):
        gep.rmsnorm(x, w, eps=-1.0)
    with pytest.raises(gep.GemmError):
        gep.rmsnorm_backward(x, x, w, rstd, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        gep.rmsnorm_backward(x, x, w, rstd, workspace=torch.empty(4, device="cuda"))
    with pytest.raises(ValueError):
        gep.rmsnorm_backward(x[:3], x, w, rstd)


@pytest.mark.parametrize("rows,cols", [(16768, 4096), (16385, 5000)])
def test_large_calls_equal_their_parts(rows, cols):
    """A call that moves more than the last-level cache holds gives, row by row, what calls on a few of
    its rows give (bit for bit), whichever kernel each of them takes."""
    announce(f"rmsnorm large {rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(rows, cols, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).bfloat16()
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    q = gep.mx_empty(rows, cols, "e4m3")
    gep.rmsnorm(x, w, residual=r, h=h, y=y, q=q, rstd=rstd)
    assert torch.equal(h, (x.float() + r.float()).bfloat16())
    values = gep.mx_dequantize(q)
    ph, py, pr = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    for a in range(0, rows, 1000):
        s = slice(a, min(a + 1000, rows))
        pq = gep.mx_empty(s.stop - a, cols, "e4m3")
        gep.rmsnorm(x[s], w, residual=r[s], h=ph[s], y=py[s], q=pq, rstd=pr[s])
        assert torch.equal(pq.codes, q.codes[s])
        assert torch.equal(gep.mx_dequantize(pq), values[s])
    assert torch.equal(ph, h) and torch.equal(py, y) and torch.equal(pr, rstd)


@pytest.mark.parametrize("rows,cols", [(16768, 4096), (16385, 5000)])
def test_large_gradients_equal_their_parts(rows, cols):
    """dx as above; dw: every row's term carries 3 u (rstd's product, dy's, the sum's), the sum (rows + 6) u
    of sum |dy n| as in test_backward."""
    announce(f"rmsnorm backward large {rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(2)
    dy, h, dres = (torch.randn(rows, cols, generator=g, device="cuda").bfloat16() for _ in range(3))
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).bfloat16()
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    dx, dw = gep.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    for a in range(0, rows, 1000):
        s = slice(a, min(a + 1000, rows))
        part, _ = gep.rmsnorm_backward(dy[s], h[s], w, rstd[s], dres=dres[s])
        assert torch.equal(part, dx[s])
    want, mag = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    for a in range(0, rows, 1000):
        s = slice(a, min(a + 1000, rows))
        t = dy[s].double() * h[s].double() * rstd[s].double()[:, None]
        want += t.sum(0)
        mag += t.abs().sum(0)
    assert ((dw.double() - want).abs() <= (rows + 6) * U * mag).all()


# (rstd is held to 2^-48 or so of itself and each product is rounded once: a y of 64 bits that lies this
# close to a border between two results may fall on either side)
EXACT = 2.0 ** -40


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [300, 1000, 5000, 17000])
def test_products_past_the_range(cols, kind):
    """h w leaves fp32's range, on either side, where h rstd w does not: y is the rounding of the
    exact product (half an fp32 step, then half a step of the type), and its codes are those of it."""
    announce(f"rmsnorm products past the range {cols} {kind}")
    g = torch.Generator().manual_seed(cols)
    scale = torch.tensor([1e37, 1e30, 1e19, 1e9, 1e5, 1.0, 1e-12, 1e-22, 1e-30, 1e-35], dtype=torch.float64)
    x = torch.randn(11, cols, generator=g, dtype=torch.float64)
    x[:10] *= scale[:, None]
    x[10] = 3e38 * x[10].sign()  # (rstd is subnormal)
    w = torch.randn(cols, generator=g, dtype=torch.float64) * 10.0 ** torch.randint(-30, 31, (cols,), generator=g).double()
    x, w = x.to(TYPES[kind]), w.to(TYPES[kind])
    h64, w64 = x.double().numpy(), w.double().numpy()
    want = h64 / np.sqrt((h64 ** 2).mean(1))[:, None] * w64
    for fmt in ("e4m3", "e2m1"):
        q, y = gep.mx_empty(11, cols, fmt), torch.empty_like(x, device="cuda")
        gep.rmsnorm(x.cuda(), w.cuda(), eps=0.0, y=y, q=q)
        check_close(y, want, U, kind, "y")
        check_mx(q, want, EXACT, fmt)
    y = gep.rmsnorm(x.cuda(), w.cuda(), eps=0.0)
    check_close(y, want, U, kind, "y alone")


@pytest.mark.parametrize("cols", [300, 5000, 17000])
def test_fp32_output_on_borders(cols):
    """Products next to the border between two codes: the fp32 y is the nearest fp32 number to each of them,
    and the codes are those of the product."""
    announce(f"rmsnorm fp32 output on borders {cols}")
    rng = np.random.RandomState(cols)
    x = torch.from_numpy(rng.randn(1, cols).astype(np.float32))
    h64 = x.double().numpy()
    r = 1 / np.sqrt((h64 ** 2).mean())
    # (numbers of five significant bits: borders of e4m3 and, some, of e2m1)
    border = rng.randint(16, 32, cols) * np.exp2(rng.randint(-6, 2, cols)) * np.sign(rng.randn(cols))
    w = (border / (h64[0] * r)).astype(np.float32)
    want = h64 * r * w.astype(np.float64)
    near = np.spacing(np.abs(want).astype(np.float32)).astype(np.float64) / 2 + EXACT * np.abs(want)
    assert (want.astype(np.float32) == border).sum() > cols // 4 and (want != border).all()
    xd, wd = x.cuda(), torch.from_numpy(w).cuda()
    for fmt in ("e4m3", "e2m1", None):
        q = gep.mx_empty(1, cols, fmt) if fmt else None
        y = torch.empty_like(xd)
        gep.rmsnorm(xd, wd, eps=0.0, y=y, q=q)
        err = np.abs(y.double().cpu().numpy() - want)
        assert (err <= near).all(), f"{fmt}: {(err > near).sum()} of {cols} are not the nearest"
        if fmt:
            check_mx(q, want, EXACT, fmt)


@pytest.mark.parametrize("kind", list(TYPES))
def test_no_rows(kind):
    """A matrix without rows gives one, with any of the outputs."""
    announce(f"rmsnorm without rows {kind}")
    x, w = torch.empty(0, 64, dtype=TYPES[kind], device="cuda"), torch.ones(64, dtype=TYPES[kind], device="cuda")
    assert gep.rmsnorm(x, w).shape == (0, 64)
    q = gep.mx_empty(0, 64, "e4m3")
    assert gep.rmsnorm(x, w, q=q) is q
    y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(0, device="cuda")
    assert gep.rmsnorm(x, w, residual=x, h=h, y=y, q=q, rstd=rstd) is y
