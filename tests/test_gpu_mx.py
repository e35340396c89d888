"""MX quantiser, its inverse and the MX product against the 64-bit implementation in mx_ref.py.

The quantiser's codes and scales are compared byte for byte. Products: every operand value is
exact, so an output differs from the 64-bit one by the order and width of the sum: at most one
fp32 half step (2^-24) of sum |a b| per added value (K of them and the C term), then half a step
of the output type. With an e4m3 operand the matrix instruction keeps the products of a block of 32
to 2^-13 of the block's largest (measured on the hardware: 1 + 2^-13 is exact, 1 + 2^-14 gives
1; e2m1 products and the sums over blocks keep all 24 bits), so each block may add 32 x 2^-13 x
max |a| max |b|; an activation passes the sum's error on with its largest slope (1.13 for GELU,
1.1 for SiLU, 1 for ReLU; 2 |x| for ReLU^2) and its own evaluation adds up to 8 fp32 steps.
"""
import sys

import numpy as np
import pytest
import torch

import gemm_epilogue_persistent_amd as gep
import mx_ref as R

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FORMATS = ["e2m1", "e4m3"]
SENTINEL = 77.0


def announce(name):
    print(f"[case] {name}", flush=True)
    sys.stdout.flush()


def values(seed, rows, cols, kind):
    """Values over many binades, with zeros, a zero block and the type's smallest and largest."""
    rng = np.random.RandomState(seed)
    x = rng.randn(rows, cols) * np.exp2(rng.randint(-6, 7, size=(rows, cols)))
    x[rng.rand(rows, cols) < 0.05] = 0.0
    x[:, : min(cols, 32)] *= 0 if rows == 2 else 1
    t = torch.from_numpy(x).to(TYPES[kind])
    f = torch.finfo(TYPES[kind])
    flat = t.view(-1)
    for i, v in enumerate((f.tiny, -f.max, f.smallest_normal / 2, -0.0)):
        if flat.numel() > 40 * (i + 1):
            flat[40 * i + 7] = v
    return t


def check_quantized(q, x64, fmt):
    codes, s = R.quantize(x64, fmt)
    nb = s.shape[1]
    got = q.codes.cpu().numpy()
    assert np.array_equal(R.load_scales(q.scales.cpu().numpy(), x64.shape[0])[:, :nb], s)
    assert (R.load_scales(q.scales.cpu().numpy(), x64.shape[0])[:, nb:] == 0).all()
    assert np.array_equal(got, R.pack(codes, fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (2, 33), (3, 8), (65, 520), (130, 1000), (127, 257), (33, 32)])
def test_quantize(rows, cols, kind, fmt):
    announce(f"quantize {rows}x{cols} {kind} {fmt}")
    x = values(rows * 7 + cols, rows, cols, kind)
    x64 = x.double().numpy()
    d = x.cuda()
    check_quantized(gep.mx_quantize(d, fmt), x64, fmt)
    # dirty storage: padding codes and scales are written
    q = gep.mx_empty(cols, rows, fmt)
    q.codes.fill_(0x55)
    q.scales.fill_(0xFF)
    assert gep.mx_quantize(d, fmt, out=q, transpose=True) is q
    check_quantized(q, x64.T, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", list(TYPES))
def test_quantize_strides(kind, fmt):
    """Row strides, odd starts, and column-contiguous inputs."""
    announce(f"quantize strides {kind} {fmt}")
    x = values(5, 70, 203, kind)
    buf = torch.full((70, 301), SENTINEL, dtype=TYPES[kind], device="cuda")
    view = buf[:, 3:206]
    view.copy_(x)
    x64 = x.double().numpy()
    check_quantized(gep.mx_quantize(view, fmt), x64, fmt)
    check_quantized(gep.mx_quantize(view, fmt, transpose=True), x64.T, fmt)
    check_quantized(gep.mx_quantize(view.t(), fmt), x64.T, fmt)
    check_quantized(gep.mx_quantize(view.t(), fmt, transpose=True), x64, fmt)
    check_quantized(gep.mx_quantize(view[:, :1], fmt), x64[:, :1], fmt)
    check_quantized(gep.mx_quantize(view[4:5], fmt, transpose=True), x64[4:5].T, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_rounding(fmt):
    """Every magnitude, every midpoint and its fp32 neighbours, under three scales, and blocks whose
    maximum lies next to a power of two."""
    announce(f"quantize rounding {fmt}")
    m = R.magnitudes(fmt)
    mid = ((m[1:] + m[:-1]) / 2).astype(np.float32)
    v = np.concatenate([m.astype(np.float32), mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9))])
    v = np.concatenate([v, -v])
    v = np.pad(v, (0, -len(v) % 31)).reshape(-1, 31)
    rows = []
    for e in (0, -100, 100):  # the first element fixes the block's scale
        rows.append(np.concatenate([np.full((len(v), 1), m[-1]), v], 1) * 2.0 ** e)
    top = np.zeros((6, 32))
    for i, a in enumerate((1.0, np.nextafter(np.float32(1), np.float32(0)), 2.0 ** -126, 2.0 ** -149, 3.4e38, 2.0 ** -130)):
        top[i, 5], top[i, 6] = a, -a / 3
    x = torch.from_numpy(np.concatenate(rows + [top]).astype(np.float32))
    x64 = x.double().numpy()
    check_quantized(gep.mx_quantize(x.cuda(), fmt), x64, fmt)
    check_quantized(gep.mx_quantize(x.t().contiguous().cuda(), fmt, transpose=True), x64, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", list(TYPES))
def test_quantize_non_finite(kind, fmt):
    """A NaN or an infinity makes its block NaN and leaves the others alone."""
    announce(f"quantize non-finite {kind} {fmt}")
    x = values(9, 40, 96, kind)
    x[3, 5], x[4, 40], x[4, 95], x[39, 64] = float("nan"), float("inf"), float("-inf"), float("nan")
    x64 = x.double().numpy()
    q = gep.mx_quantize(x.cuda(), fmt)
    check_quantized(q, x64, fmt)
    check_quantized(gep.mx_quantize(x.cuda(), fmt, transpose=True), x64.T, fmt)
    v = gep.mx_dequantize(q, dtype=torch.float32).cpu()
    bad = torch.zeros(40, 3, dtype=torch.bool)
    bad[3, 0] = bad[4, 1] = bad[4, 2] = bad[39, 2] = True
    assert torch.equal(v.view(40, 3, 32).isnan().all(-1), bad) and torch.equal(v.view(40, 3, 32).isnan().any(-1), bad)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,k", [(1, 1), (3, 40), (66, 515), (5, 4096)])
def test_dequantize(rows, k, kind, fmt):
    announce(f"dequantize {rows}x{k} {kind} {fmt}")
    rng = np.random.RandomState(k)
    nb = -(-k // 32)
    codes = rng.randint(0, 16 if fmt == "e2m1" else 256, size=(rows, nb * 32))
    s = rng.randint(100, 130, size=(rows, nb))
    s[0, 0] = {"f16": 120, "bf16": 0, "f32": 0}[kind]
    if nb > 2:
        s[-1, 2] = 255
    q = gep.MxTensor(torch.from_numpy(R.pack(codes, fmt)).cuda(), torch.from_numpy(R.store_scales(s, 9)).cuda(), fmt, k)
    want = torch.from_numpy(R.values(codes, s, fmt, k)).float().to(TYPES[kind])
    buf = torch.full((rows, k + 3), SENTINEL, dtype=TYPES[kind], device="cuda")
    got = gep.mx_dequantize(q, out=buf[:, :k])
    assert torch.equal(got.cpu().isnan(), want.isnan())
    assert torch.equal(got.cpu().nan_to_num(), want.nan_to_num())
    assert (buf[:, k:] == SENTINEL).all()


# ---- products

def operand(seed, rows, k, fmt, spread=3):
    """Random codes (no NaN code) and scales; stored tensor and 64-bit values."""
    rng = np.random.RandomState(seed)
    nb = -(-k // 32)
    codes = rng.randint(0, 16 if fmt == "e2m1" else 256, size=(rows, nb * 32))
    if fmt == "e4m3":
        codes = np.where((codes & 127) == 127, 0, codes)
        codes = np.where((codes & 127) > 0x50, codes & ~0x20, codes)  # (keep the magnitudes moderate)
    codes[:, k:] = 0
    s = rng.randint(127 - spread, 128 + spread, size=(rows, nb))
    return codes, s


def stored(codes, s, fmt, k):
    # scales of rows past the end hold NaN bytes: they must not matter
    return gep.MxTensor(torch.from_numpy(R.pack(codes, fmt)).cuda(), torch.from_numpy(R.store_scales(s, 255)).cuda(), fmt, k)


SLOPE = {"none": 1.0, "relu": 1.0, "gelu_tanh": 1.13, "silu": 1.1}


def check_product(got, want, bound, kind, act="none", pre=None):
    g = got.double().cpu().numpy()
    assert g.shape == want.shape
    eps = torch.finfo(TYPES[kind]).eps / 2
    if act == "relu_sq":
        bound = 2 * (np.abs(pre) + bound) * bound
    else:
        bound = SLOPE[act] * bound
    if act != "none":
        bound = bound + 2.0 ** -20 * (np.abs(want) + (np.abs(pre) if act in ("gelu_tanh", "silu") else 0))
    err = np.abs(g - want)
    tol = bound * (1 + eps) + eps * np.abs(want) + torch.finfo(TYPES[kind]).tiny
    assert np.isfinite(g).all()
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} out, worst {np.max(err / np.maximum(tol, 1e-300)):.3g}"


def guarded(M, N, kind):
    buf = torch.full((M + 1, N + 16), SENTINEL, dtype=TYPES[kind], device="cuda")
    return buf[:M, :N], buf


def untouched(buf, M, N):
    return bool((buf[M:] == SENTINEL).all()) and bool((buf[:, N:] == SENTINEL).all())


def largest(v):
    """The largest magnitude of each block of 32 (rows, blocks)."""
    return np.abs(R.blocks(v)).max(-1)


def run_product(M, N, K, fa, fb, tile, c=None, d="f32", post=None, act="none", sizes=None, seed=0, scale=1.0, split=1):
    ca, sa = operand(seed + 1, M, K, fa)
    va = R.values(ca, sa, fa, K)
    G = len(sizes) if sizes is not None else None
    a = stored(ca, sa, fa, K)
    cu = None
    if G is None:
        cb, sb = operand(seed + 2, N, K, fb)
        b = stored(cb, sb, fb, K)
        vb = R.values(cb, sb, fb, K)
        x, mag, mx = va @ vb.T, np.abs(va) @ np.abs(vb).T, largest(va) @ largest(vb).T
    else:
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        parts = [operand(seed + 10 + g, N, K, fb) for g in range(G)]
        bs = [stored(p, q, fb, K) for p, q in parts]
        b = gep.MxTensor(torch.stack([t.codes for t in bs]), torch.stack([t.scales for t in bs]), fb, K)
        cu = torch.from_numpy(off).cuda()
        x, mag, mx = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
        for g in range(G):
            r = slice(off[g], off[g + 1])
            vb = R.values(*parts[g], fb, K)
            x[r], mag[r], mx[r] = va[r] @ vb.T, np.abs(va[r]) @ np.abs(vb).T, largest(va[r]) @ largest(vb).T
    C = None
    if c is not None:
        C, cbuf = guarded(M, N, c)
        C.copy_(torch.randn(M, N, generator=torch.Generator().manual_seed(seed)).mul(scale))
        x = x + C.double().cpu().numpy()
        mag = mag + np.abs(C.double().cpu().numpy())
    D, dbuf = guarded(M, N, d) if d else (None, None)
    P, pbuf = guarded(M, N, post) if post else (None, None)
    plan = gep.MxPlan(a, b, C, D, P, act=act, cu_seqlens_m=cu, tile=tile, split=split)
    assert split == 1 or (plan.tile()[1] > 1) == (K > 512)
    plan.run(a, b, C, D, P, cu_seqlens_m=cu)
    torch.cuda.synchronize()
    bound = (K + 1) * 2.0 ** -24 * mag
    if "e4m3" in (fa, fb):
        bound = bound + 32 * 2.0 ** -13 * mx
    for buf in (dbuf, pbuf):
        assert buf is None or untouched(buf, M, N)
    if D is not None:
        check_product(D, x, bound, d)
    if P is not None:
        check_product(P, R.act(x, act), bound, post, act, x)


TILES = ["256", "128", "32x64", "32", "16x32", "16"]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("fa", FORMATS)
@pytest.mark.parametrize("fb", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 8, 1), (17, 40, 33), (130, 264, 160), (70, 520, 1000), (300, 136, 2100)])
def test_product(M, N, K, fa, fb, tile):
    announce(f"product {M}x{N}x{K} {fa} x {fb} tile {tile}")
    run_product(M, N, K, fa, fb, tile)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("K", [32, 128, 256, 384, 512, 640, 1024, 4128])
def test_product_depths(K, tile):
    """Every number of steps modulo the loops' unrolling."""
    announce(f"product depth {K} tile {tile}")
    run_product(40, 72, K, "e4m3", "e2m1", tile, seed=K)
    run_product(24, 72, K, "e2m1", "e2m1", tile, seed=K + 1)


@pytest.mark.parametrize("tile", TILES[1:])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e2m1"), ("e2m1", "e2m1"), ("e4m3", "e4m3")])
@pytest.mark.parametrize("M,N,K,split", [(1, 8, 520, 2), (70, 136, 1000, 2), (150, 264, 2100, 5), (33, 72, 4128, 9), (40, 40, 500, 4)])
def test_product_split_k(M, N, K, split, fa, fb, tile):
    announce(f"product split K {M}x{N}x{K} / {split} {fa} x {fb} tile {tile}")
    run_product(M, N, K, fa, fb, tile, c="bf16", d="f32", post="bf16", act="silu", split=split, seed=31)


@pytest.mark.parametrize("fa", FORMATS)
@pytest.mark.parametrize("sizes", [None, [1000, 0, 3097, 253]])
def test_product_split_tail(sizes, fa):
    """More 256x256 tiles than one round of the card, the last round a small one."""
    announce(f"product split tail {fa} {sizes}")
    run_product(4350, 4104, 96, fa, "e2m1", "256", sizes=sizes, seed=21, d="bf16")


@pytest.mark.parametrize("tile", TILES)
def test_product_exact(tile):
    """Small integers under scale 1: every partial sum is exact, so is the result."""
    announce(f"product exact tile {tile}")
    M, N, K = 150, 296, 768
    rng = np.random.RandomState(3)
    for fa, fb in (("e2m1", "e2m1"), ("e4m3", "e2m1"), ("e4m3", "e4m3"), ("e2m1", "e4m3")):
        va, vb = rng.randint(-4, 5, size=(M, K)).astype(float), rng.randint(-3, 4, size=(N, K)).astype(float)
        one = {"e2m1": 127 + 2 - 2, "e4m3": 127}
        ca, sa = R.quantize(va, fa)
        cb, sb = R.quantize(vb, fb)
        a, b = stored(ca, sa, fa, K), stored(cb, sb, fb, K)
        D = torch.empty(M, N, device="cuda")
        gep.mx_gemm(a, b, D, tile=tile)
        want = R.values(ca, sa, fa, K) @ R.values(cb, sb, fb, K).T
        assert np.array_equal(D.double().cpu().numpy(), want), (fa, fb, one)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("c,d,post,act", [
    (None, "bf16", None, "none"), ("bf16", "bf16", "bf16", "silu"), (None, None, "f16", "gelu_tanh"),
    ("f32", "f16", "f32", "relu"), ("f16", None, "f32", "relu_sq"), (None, "f16", "bf16", "none")])
def test_product_epilogue(c, d, post, act, tile):
    announce(f"product epilogue c={c} d={d} post={post} {act} tile {tile}")
    # (values small enough for f16)
    run_product(66, 136, 64, "e2m1", "e2m1", tile, c, d, post, act, seed=11)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("sizes", [[5], [0, 3, 0, 70, 1, 0], [130, 0, 257, 16], [0] * 70 + [9, 0, 40] + [0] * 3, [1] * 33])
def test_product_grouped(sizes, tile):
    announce(f"product grouped {sizes} tile {tile}")
    run_product(sum(sizes), 72, 160, "e4m3", "e2m1", tile, sizes=sizes, seed=5, d="bf16", post="bf16", act="silu")


@pytest.mark.parametrize("tile", TILES)
def test_product_grouped_malformed(tile):
    """Offsets that do not run 0 .. M without decreasing write nothing."""
    announce(f"product grouped malformed tile {tile}")
    q = gep.mx_quantize(torch.randn(20, 64, device="cuda"), "e4m3")
    b = gep.mx_empty(16, 64, "e4m3", groups=2)
    b.codes.zero_()
    for bad in ([0, 30, 20], [1, 10, 20], [0, 10, 19], [0, -5, 20], [0, 10, 2 ** 31 - 1]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        D = torch.full((20, 16), SENTINEL, device="cuda")
        gep.MxPlan(q, b, None, D, cu_seqlens_m=cu, tile=tile).run(q, b, None, D, cu_seqlens_m=cu)
        assert (D == SENTINEL).all(), bad


@pytest.mark.parametrize("tile", TILES)
def test_product_empty_k_and_rows(tile):
    announce(f"product empty tile {tile}")
    a, b = gep.mx_empty(20, 0, "e4m3"), gep.mx_empty(24, 0, "e2m1")
    C = torch.randn(20, 24, device="cuda")
    D = torch.full((20, 24), SENTINEL, device="cuda")
    gep.mx_gemm(a, b, D, C, tile=tile)
    assert torch.equal(D, C)
    gep.mx_gemm(a, b, D, tile=tile)
    assert (D == 0).all()
    a, b = gep.mx_empty(0, 64, "e4m3"), gep.mx_empty(24, 64, "e2m1")
    assert gep.mx_gemm(a, b, tile=tile).shape == (0, 24)


@pytest.mark.parametrize("tile", TILES)
def test_product_nan_scale(tile):
    """A NaN block makes the outputs of its row NaN, and only those."""
    announce(f"product NaN scale tile {tile}")
    x = torch.randn(50, 600, device="cuda")
    x[21, 555] = float("nan")
    a, b = gep.mx_quantize(x, "e4m3"), gep.mx_quantize(torch.randn(40, 600, device="cuda"), "e2m1")
    D = gep.mx_gemm(a, b, tile=tile)
    assert D[21].isnan().all() and D.isnan().any(1).sum() == 1


def test_product_in_place_and_stream():
    """C may be D itself; a plan runs on the stream it is given, and repeats bit for bit."""
    announce("product in place, other stream")
    a = gep.mx_quantize(torch.randn(100, 500, device="cuda"), "e4m3")
    b = gep.mx_quantize(torch.randn(64, 500, device="cuda"), "e4m3")
    C = torch.randn(100, 64, device="cuda")
    want = gep.mx_gemm(a, b, torch.empty_like(C), C)
    D = C.clone()
    plan = gep.MxPlan(a, b, D, D)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan.run(a, b, D, D, stream=s)
    s.synchronize()
    assert torch.equal(D, want)
    split = gep.MxPlan(a, gep.mx_empty(64, 500, "e4m3"), None, D, split=2)
    assert split.tile()[1] == 1 and split.workspace_bytes == 0  # one scale tile cannot be shared out
    with pytest.raises(ValueError):
        plan.run(a, b, D, D.t())
    with pytest.raises(ValueError):
        plan.run(a, b, None, D)


def test_workspace():
    """A given workspace is used; one that is too small is refused; without one in the C ABI K is
    not split; runs repeat bit for bit."""
    announce("product workspace")
    import ctypes
    from gemm_epilogue_persistent_amd import _abi
    a = gep.mx_quantize(torch.randn(40, 2048, device="cuda"), "e4m3")
    b = gep.mx_quantize(torch.randn(64, 2048, device="cuda"), "e4m3")
    D, E = torch.empty(40, 64, device="cuda"), torch.empty(40, 64, device="cuda")
    plan = gep.MxPlan(a, b, None, D, tile="32", split=4)
    assert plan.workspace_bytes == 4 * 40 * 64 * 4
    plan.run(a, b, None, D)
    ws = torch.full((plan.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")
    plan.run(a, b, None, E, workspace=ws)
    assert torch.equal(D, E)
    assert torch.equal(ws.view(torch.float32).view(4, 40, 64).double().sum(0).float(), E) or (
        (ws.view(torch.float32).view(4, 40, 64).sum(0) - E).abs().max() <= 1e-5 * E.abs().max())
    with pytest.raises(gep.GemmError):
        plan.run(a, b, None, E, workspace=ws[:-16])
    with pytest.raises(gep.GemmError):
        plan.run(a, b, None, E, workspace=torch.empty(plan.workspace_bytes + 16, dtype=torch.uint8, device="cuda")[8:])
    with pytest.raises(ValueError):
        plan.run(a, b, None, E, workspace=ws.float())
    args = _abi.MxGemmArgs(a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(), b.scales.data_ptr(), None,
                           E.data_ptr(), None, None, None, 0)
    E.zero_()
    _abi.check(_abi.load().mx_gemm_run(plan.handle, ctypes.byref(args), torch.cuda.current_stream().cuda_stream))
    want = gep.mx_gemm(a, b, torch.empty_like(E), tile="32", split=1)
    assert torch.equal(E, want)


def test_python_refusals():
    a = gep.mx_empty(16, 64, "e4m3")
    b = gep.mx_empty(24, 64, "e2m1")
    D = torch.empty(16, 24, device="cuda")
    g = gep.mx_empty(24, 64, "e2m1", groups=2)
    cu = torch.tensor([0, 4, 16], dtype=torch.int32, device="cuda")
    for args, kw in (((a, gep.mx_empty(24, 96, "e2m1"), None, D), {}), ((a, g, None, D), {}),
                     ((a, b, None, D), dict(cu_seqlens_m=cu)), ((a, g, None, D), dict(cu_seqlens_m=cu[:2])),
                     ((a, g, None, D), dict(cu_seqlens_m=cu.long())), ((a, b, None, D[:8]), {}),
                     ((a, b, None, D), dict(act="tanh")), ((a, b, None, D), dict(tile="512")),
                     ((a, b, None, D.t().contiguous().t()), {})):
        with pytest.raises(ValueError):
            gep.MxPlan(*args, **kw)
    with pytest.raises(TypeError):
        gep.MxPlan(a, b, None, D.double())
    with pytest.raises(gep.GemmError):
        gep.MxPlan(a, b)
    with pytest.raises(gep.GemmError):
        gep.MxPlan(a, gep.mx_empty(20, 64, "e2m1"), None, torch.empty(16, 20, device="cuda"))
    x = torch.zeros(16, 64, device="cuda")
    with pytest.raises(ValueError):
        gep.mx_quantize(x, "e4m3", out=b)
    with pytest.raises(ValueError):
        gep.mx_quantize(x, "e2m1", out=a)
    with pytest.raises(ValueError):
        gep.mx_quantize(x[:, ::2], "e2m1")
    with pytest.raises(ValueError):
        gep.mx_quantize(x.expand(2, 16, 64)[:, 0].as_strided((4, 64), (0, 1)), "e2m1")
    with pytest.raises(TypeError):
        gep.mx_quantize(x.double(), "e2m1")
    with pytest.raises(ValueError):
        gep.mx_dequantize(a, out=torch.empty(16, 63, device="cuda"))
    with pytest.raises(ValueError):
        gep.mx_dequantize(g)


@pytest.mark.parametrize("tile", ["256", "128"])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e2m1"), ("e2m1", "e2m1"), ("e4m3", "e4m3")])
@pytest.mark.parametrize("c,d,post,act", [
    ("bf16", "bf16", None, "none"), ("f16", None, "bf16", "silu"), (None, "bf16", "f16", "gelu_tanh"),
    ("bf16", "f16", "bf16", "silu"), ("f32", "bf16", "bf16", "relu")])
def test_product_epilogue_over_tiles(c, d, post, act, fa, fb, tile):
    """Several tiles a workgroup and edges in both directions: the stores of one tile under the first
    transfers of the next, with each kind of epilogue."""
    announce(f"product epilogue over tiles c={c} d={d} post={post} {act} {fa} x {fb} tile {tile}")
    if "e4m3" in (fa, fb):  # (products of these operands pass f16's largest value, the first here with 67016)
        d, post = ("bf16" if t == "f16" else t for t in (d, post))
    n = 5640 if tile == "256" else 2312  # (414 and 608 tiles; a last round of more than half the card is not split)
    run_product(4400 if tile == "256" else 4000, n, 160, fa, fb, tile, c, d, post, act, seed=41)


@pytest.mark.parametrize("fa,fb", [("e4m3", "e2m1"), ("e2m1", "e2m1"), ("e4m3", "e4m3")])
def test_product_epilogue_over_deep_tiles(fa, fb):
    announce(f"product epilogue over deep tiles {fa} x {fb}")
    run_product(4400, 5640, 1000, fa, fb, "256", "bf16", "bf16", "bf16", "silu", seed=45)


@pytest.mark.parametrize("fa", FORMATS)
@pytest.mark.parametrize("c,d,post", [("bf16", "bf16", None), (None, "bf16", "bf16"), ("bf16", "bf16", "bf16")])
def test_product_epilogue_over_grouped_tiles(c, d, post, fa):
    announce(f"product epilogue over grouped tiles c={c} d={d} post={post} {fa}")
    run_product(4400, 5640, 96, fa, "e2m1", "256", c, d, post, "silu" if post else "none", sizes=[1000, 0, 3147, 253], seed=43)


@pytest.mark.parametrize("tile", ["256", "128", "32"])
def test_product_c_in_place(tile):
    """C in the place of D, and of PostAct."""
    announce(f"product C in place tile {tile}")
    a = gep.mx_quantize(torch.randn(700, 200, device="cuda"), "e4m3")
    b = gep.mx_quantize(torch.randn(520, 200, device="cuda"), "e2m1")
    C = torch.randn(700, 520, device="cuda").bfloat16()
    D, P = torch.empty_like(C), torch.empty_like(C)
    gep.mx_gemm(a, b, D, C, P, act="silu", tile=tile)
    x = C.clone()
    gep.mx_gemm(a, b, x, x, None, tile=tile)
    assert torch.equal(x, D)
    x, y = C.clone(), C.clone()
    gep.mx_gemm(a, b, None, x, x, act="silu", tile=tile)
    assert torch.equal(x, P)
    gep.mx_gemm(a, b, y, y, x, act="silu", tile=tile)
    assert torch.equal(y, D) and torch.equal(x, P)


def test_product_aliases_refused():
    a, b = gep.mx_empty(16, 64, "e4m3"), gep.mx_empty(24, 64, "e2m1")
    buf = torch.zeros(16, 64, device="cuda")
    for C, D, P in ((buf[:, :24], buf.view(32, 32)[:16, :24], None), (buf[:, :24], torch.empty(16, 24, device="cuda"), buf.view(32, 32)[:16, :24]),
                    (None, buf[:, :24], buf[:, :24]), (buf.bfloat16()[:, :24], buf[:, :24], buf[:, :24])):
        with pytest.raises(gep.GemmError):
            gep.mx_gemm(a, b, D, C, P, act="silu" if P is not None else "none")
