"""8-bit matrices with a scale per 128 values: the quantiser, its inverse and the product against the 64-bit
implementation in fp8_ref.py.

The quantiser's codes and scales are compared byte for byte. Products: an operand value is code * scale. Within
a block the matrix instruction keeps the products of 32 values to 2^-13 of their largest, so that each
block of 128 may be off by 128 x 2^-13 x max |a| max |b|; the scales' product, the FMA of each block (and, where a
column has its own scale, one product more) round to fp32, each by 2^-24 of what is summed so far; then
the sums of slices and C, and half a step of the output type. An activation passes the sum's error on with its
largest slope (1.13 for GELU, 1.1 for SiLU, 1 for ReLU; 2 |x| for ReLU^2) and its own evaluation adds up to 16
fp32 steps.
"""
import sys

import numpy as np
import pytest
import torch

import fp8_ref as R
import gemm_epilogue_persistent_amd as gep

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SENTINEL = 77.0
SIZES = [(1, 1), (1, 4096), (2, 33), (3, 8), (65, 520), (130, 1000), (127, 257), (33, 128), (257, 16), (128, 128), (300, 135)]


def announce(name):
    print(f"[case] {name}", flush=True)
    sys.stdout.flush()


def values(seed, rows, cols, kind):
    """Values over many binades, with zeros, zero blocks and the type's smallest and largest."""
    rng = np.random.RandomState(seed)
    x = rng.randn(rows, cols) * np.exp2(rng.randint(-6, 7, size=(rows, cols)))
    x[rng.rand(rows, cols) < 0.05] = 0.0
    if rows > 4:
        x[3] = 0.0
        x[:, cols // 2] = 0.0
    t = torch.from_numpy(x).to(TYPES[kind])
    f = torch.finfo(TYPES[kind])
    flat = t.view(-1)
    for i, v in enumerate((f.tiny, -f.max, f.smallest_normal / 2, -0.0)):
        if flat.numel() > 400 * (i + 1):
            flat[400 * i + 7] = v
    return t


def check_quantized(q, x64, tiles=False):
    codes, s = R.quantize(x64, tiles)
    nb = s.shape[1]
    got = R.load_scales(q.scales.cpu().numpy(), x64.shape[0], tiles)
    assert np.array_equal(got[:, :nb], s, equal_nan=True)
    assert (got[:, nb:] == 0).all()
    assert np.array_equal(q.codes.cpu().numpy(), codes)


def dirty(rows, cols, tiles=False):
    """Storage whose padding must be written."""
    q = gep.fp8_empty(rows, cols, tiles=tiles)
    q.codes.fill_(0x55)
    q.scales.fill_(float("nan"))
    return q


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize(rows, cols, kind):
    announce(f"fp8 quantize {rows}x{cols} {kind}")
    x = values(rows * 7 + cols, rows, cols, kind)
    x64, d = x.double().numpy(), x.cuda()
    q = dirty(rows, cols)
    assert gep.fp8_quantize(d, out=q) is q
    check_quantized(q, x64)
    q, qt = dirty(rows, cols), dirty(cols, rows)
    assert gep.fp8_quantize(d, out=q, out_t=qt) is q
    check_quantized(q, x64)
    check_quantized(qt, x64.T)
    qt = dirty(cols, rows)
    assert gep.fp8_quantize(d, out_t=qt) is qt
    check_quantized(qt, x64.T)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_tiles(rows, cols, kind):
    announce(f"fp8 quantize tiles {rows}x{cols} {kind}")
    x = values(rows * 5 + cols, rows, cols, kind)
    x64, d = x.double().numpy(), x.cuda()
    check_quantized(gep.fp8_quantize(d, tiles=True), x64, True)
    q, qt = dirty(rows, cols, True), dirty(cols, rows, True)
    gep.fp8_quantize(d, out=q, out_t=qt)
    check_quantized(q, x64, True)
    check_quantized(qt, x64.T, True)
    qt = dirty(cols, rows, True)
    gep.fp8_quantize(d, out_t=qt)
    check_quantized(qt, x64.T, True)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
def test_quantize_strides(kind, tiles):
    """Row strides, odd starts, and column-contiguous inputs."""
    announce(f"fp8 quantize strides {kind}")
    x = values(5, 170, 203, kind)
    buf = torch.full((170, 301), SENTINEL, dtype=TYPES[kind], device="cuda")
    view = buf[:, 3:206]
    view.copy_(x)
    x64 = x.double().numpy()
    for v, w in ((view, x64), (view.t(), x64.T), (view[:, :1], x64[:, :1]), (view[4:5], x64[4:5])):
        check_quantized(gep.fp8_quantize(v, tiles=tiles), w, tiles)
        qt = dirty(w.shape[1], w.shape[0], tiles)
        gep.fp8_quantize(v, out_t=qt)
        check_quantized(qt, w.T, tiles)


@pytest.mark.parametrize("kind", list(TYPES))
def test_quantize_rounding(kind):
    """Blocks of every largest magnitude of 8 bits with every 16-bit neighbour of every border between two codes
    (fp32: the exact borders' neighbours under factors of 13 bits), and the ends of the range."""
    announce(f"fp8 quantize rounding {kind}")
    m = R.magnitudes()
    mid = (m[1:] + m[:-1]) / 2
    rows = []
    for a in range(128, 256):
        top = a / 128.0
        r = R.factor(np.array([top]))[0]
        v = torch.from_numpy(mid / r).to(TYPES[kind]).double().numpy()
        near = [v]
        for d in (-1, 1):
            t = torch.from_numpy(v).to(TYPES[kind])
            bits = t.view(torch.int32 if kind == "f32" else torch.int16)
            near.append((bits + d).view(TYPES[kind]).double().numpy())
        v = np.concatenate(near)
        v = np.pad(v, (0, -len(v) % 127)).reshape(-1, 127)
        rows.append(np.concatenate([np.full((len(v), 1), top), v * np.where(np.arange(127) % 2, 1, -1)], 1))
    x = np.concatenate(rows)
    x = np.where(np.abs(x) > x[:, :1], 0, x)
    scale = {"f16": (1,), "bf16": (1, 2.0 ** -100, 2.0 ** 100), "f32": (1, 2.0 ** -100, 2.0 ** 100)}[kind]
    x = torch.from_numpy(np.concatenate([x * s for s in scale])).to(TYPES[kind])
    x64 = x.double().numpy()
    q, qt = dirty(*x.shape), dirty(*x.shape[::-1])
    gep.fp8_quantize(x.cuda(), out=q, out_t=qt)
    check_quantized(q, x64)
    check_quantized(qt, x64.T)
    ends = torch.zeros(8, 128, dtype=TYPES[kind])
    f = torch.finfo(TYPES[kind])
    for i, v in enumerate((f.max, f.tiny, f.smallest_normal / 4, f.eps, 448.0, 1.0, -f.max, 3 * f.tiny)):
        ends[i, 5], ends[i, 6] = v, -v / 3
    check_quantized(gep.fp8_quantize(ends.cuda()), ends.double().numpy())


def test_quantize_random_fp32():
    """Random fp32 values: products with the factor that need more than 24 bits."""
    announce("fp8 quantize random fp32")
    x = torch.randn(700, 1000, generator=torch.Generator().manual_seed(3))
    check_quantized(gep.fp8_quantize(x.cuda()), x.double().numpy())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("tiles", [False, True])
def test_quantize_not_finite(kind, tiles):
    announce(f"fp8 quantize not finite {kind}")
    x = values(9, 300, 400, kind)
    x[5, 7], x[260, 300], x[131, 399] = float("inf"), float("nan"), -float("inf")
    x64 = x.double().numpy()
    q, qt = dirty(300, 400, tiles), dirty(400, 300, tiles)
    gep.fp8_quantize(x.cuda(), out=q, out_t=qt)
    check_quantized(q, x64, tiles)
    check_quantized(qt, x64.T, tiles)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("rows,k", [(1, 1), (5, 200), (130, 1000), (257, 16)])
def test_dequantize(rows, k, tiles, kind):
    announce(f"fp8 dequantize {rows}x{k} {kind}")
    codes, s = operand(rows + k, rows, k, tiles)
    q = stored(codes, s, k, tiles)
    buf = torch.full((rows, k + 9), SENTINEL, dtype=TYPES[kind], device="cuda")
    out = buf[:, 3:3 + k]
    gep.fp8_dequantize(q, out=out)
    v = R.values(codes, s, k, tiles)
    # (the product is rounded to fp32, then to the type)
    want = torch.from_numpy(v.astype(np.float32)).to(TYPES[kind])
    assert torch.equal(out.cpu(), want)
    assert (buf[:, :3] == SENTINEL).all() and (buf[:, 3 + k:] == SENTINEL).all()


def operand(seed, rows, k, tiles=False):
    """Random codes and scales."""
    rng = np.random.RandomState(seed)
    codes = np.zeros((rows, -(-k // 16) * 16), np.uint8)
    c = rng.randint(0, 256, size=(rows, k))
    c[(c & 127) == 127] -= 1
    c[rng.rand(rows, k) < 0.3] &= 0xBF  # (smaller exponents, and with them sums that do not hang on one value)
    codes[:, :k] = c
    s = np.exp2(rng.randint(-8, 3, size=(-(-rows // 128) if tiles else rows, -(-k // 128)))) * rng.uniform(1, 2) / 448
    return codes, (s * rng.uniform(1, 2, size=s.shape)).astype(np.float32)


def stored(codes, s, k, tiles=False):
    # scales of rows past the end are NaN: they must not matter
    return gep.Fp8Tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(R.store_scales(s, tiles, np.nan)).cuda(), k)


SLOPE = {"none": 1.0, "relu": 1.0, "gelu_tanh": 1.13, "silu": 1.1}


def check_product(got, want, bound, kind, act="none", pre=None):
    g = got.double().cpu().numpy()
    assert g.shape == want.shape
    eps = torch.finfo(TYPES[kind]).eps / 2
    bound = 2 * (np.abs(pre) + bound) * bound if act == "relu_sq" else SLOPE[act] * bound
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
    """The largest magnitude of each block of 128 (rows, blocks)."""
    rows, k = v.shape
    b = np.zeros((rows, -(-k // 128) * 128))
    b[:, :k] = np.abs(v)
    return b.reshape(rows, b.shape[1] // 128, 128).max(-1)


def run_product(M, N, K, tile, tiles=True, c=None, d="f32", post=None, act="none", sizes=None, seed=0, split=1):
    ca, sa = operand(seed + 1, M, K)
    va = R.values(ca, sa, K)
    G = len(sizes) if sizes is not None else None
    a, cu = stored(ca, sa, K), None
    if G is None:
        cb, sb = operand(seed + 2, N, K, tiles)
        b = stored(cb, sb, K, tiles)
        vb = R.values(cb, sb, K, tiles)
        x, mag, mx = va @ vb.T, np.abs(va) @ np.abs(vb).T, largest(va) @ largest(vb).T
    else:
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        parts = [operand(seed + 10 + g, N, K, tiles) for g in range(G)]
        bs = [stored(*p, K, tiles) for p in parts]
        b = gep.Fp8Tensor(torch.stack([t.codes for t in bs]), torch.stack([t.scales for t in bs]), K)
        cu = torch.from_numpy(off).cuda()
        x, mag, mx = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
        for g in range(G):
            r = slice(off[g], off[g + 1])
            vb = R.values(*parts[g], K, tiles)
            x[r], mag[r], mx[r] = va[r] @ vb.T, np.abs(va[r]) @ np.abs(vb).T, largest(va[r]) @ largest(vb).T
    C = None
    if c is not None:
        C, cbuf = guarded(M, N, c)
        C.copy_(torch.randn(M, N, generator=torch.Generator().manual_seed(seed)))
        x = x + C.double().cpu().numpy()
        mag = mag + np.abs(C.double().cpu().numpy())
    D, dbuf = guarded(M, N, d) if d else (None, None)
    P, pbuf = guarded(M, N, post) if post else (None, None)
    plan = gep.Fp8Plan(a, b, C, D, P, act=act, cu_seqlens_m=cu, tile=tile, split=split)
    assert split == 1 or (plan.tile()[1] > 1) == (K > 512)
    plan.run(a, b, C, D, P, cu_seqlens_m=cu)
    torch.cuda.synchronize()
    # four roundings a block, and the joins of up to 64 slices and eight waves
    bound = (4 * (-(-K // 128)) + 74) * 2.0 ** -24 * mag + 128 * 2.0 ** -13 * mx
    for buf in (dbuf, pbuf):
        assert buf is None or untouched(buf, M, N)
    if D is not None:
        check_product(D, x, bound, d)
    if P is not None:
        check_product(P, R.act(x, act), bound, post, act, x)


TILES = ["256", "128", "64", "32", "16x32", "16"]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("M,N,K", [(1, 8, 1), (17, 40, 33), (130, 264, 160), (70, 520, 1000), (300, 136, 2100)])
def test_product(M, N, K, tiles, tile):
    announce(f"fp8 product {M}x{N}x{K} {'tiles' if tiles else 'rows'} tile {tile}")
    run_product(M, N, K, tile, tiles)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("K", [16, 128, 256, 384, 512, 640, 1024, 4128])
def test_product_depths(K, tiles, tile):
    """Every number of steps modulo the loops' unrolling."""
    announce(f"fp8 product depth {K} tile {tile}")
    run_product(40, 72, K, tile, tiles, seed=K)


@pytest.mark.parametrize("tile", TILES[1:])
@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("M,N,K,split", [(1, 8, 520, 2), (70, 136, 1000, 2), (150, 264, 2100, 5), (33, 72, 4128, 9), (40, 40, 500, 4)])
def test_product_split_k(M, N, K, split, tiles, tile):
    announce(f"fp8 product split K {M}x{N}x{K} / {split} tile {tile}")
    run_product(M, N, K, tile, tiles, c="bf16", d="f32", post="bf16", act="silu", split=split, seed=31)


@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("sizes", [None, [1000, 0, 3097, 253]])
def test_product_split_tail(sizes, tiles):
    """More 256x256 tiles than one round of the card, the last round a small one."""
    announce(f"fp8 product split tail {sizes}")
    run_product(4350, 4104, 96, "256", tiles, sizes=sizes, seed=21, d="bf16")


@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("tile", TILES)
def test_product_exact(tile, tiles):
    """Small integers under scales that are powers of two: every partial sum is exact, so is the result; each block
    has scales of its own, so that none is taken for another's."""
    announce(f"fp8 product exact tile {tile}")
    M, N, K = 150, 296, 1400
    rng = np.random.RandomState(3)

    def integers(rows, k, t):
        m = R.magnitudes()
        v = rng.randint(-4, 5, size=(rows, k))
        codes = np.zeros((rows, -(-k // 16) * 16), np.uint8)
        codes[:, :k] = np.searchsorted(m, np.abs(v)) | np.where(v < 0, 128, 0)
        return codes, np.exp2(rng.randint(-2, 3, size=(-(-rows // 128) if t else rows, -(-k // 128)))).astype(np.float32)

    (ca, sa), (cb, sb) = integers(M, K, False), integers(N, K, tiles)
    D = torch.empty(M, N, device="cuda")
    gep.fp8_gemm(stored(ca, sa, K), stored(cb, sb, K, tiles), D, tile=tile)
    want = R.values(ca, sa, K) @ R.values(cb, sb, K, tiles).T
    assert np.array_equal(D.double().cpu().numpy(), want)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("c,d,post,act", [
    (None, "bf16", None, "none"), ("bf16", "bf16", "bf16", "silu"), (None, None, "f16", "gelu_tanh"),
    ("f32", "f16", "f32", "relu"), ("f16", None, "f32", "relu_sq"), (None, "f16", "bf16", "none")])
def test_product_epilogue(c, d, post, act, tile):
    announce(f"fp8 product epilogue c={c} d={d} post={post} {act} tile {tile}")
    run_product(66, 136, 64, tile, True, c, d, post, act, seed=11)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("sizes", [[5], [0, 3, 0, 70, 1, 0], [130, 0, 257, 16], [0] * 70 + [9, 0, 40] + [0] * 3, [1] * 33])
def test_product_grouped(sizes, tiles, tile):
    announce(f"fp8 product grouped {sizes} tile {tile}")
    run_product(sum(sizes), 136, 160, tile, tiles, sizes=sizes, seed=5, d="bf16", post="bf16", act="silu")


@pytest.mark.parametrize("tile", TILES)
def test_product_grouped_malformed(tile):
    """Offsets that do not run 0 .. M without decreasing write nothing."""
    announce(f"fp8 product grouped malformed tile {tile}")
    q = gep.fp8_quantize(torch.randn(20, 64, device="cuda"))
    b = gep.fp8_empty(16, 64, tiles=True, groups=2)
    b.codes.zero_()
    for bad in ([0, 30, 20], [1, 10, 20], [0, 10, 19], [0, -5, 20], [0, 10, 2 ** 31 - 1]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        D = torch.full((20, 16), SENTINEL, device="cuda")
        gep.Fp8Plan(q, b, None, D, cu_seqlens_m=cu, tile=tile).run(q, b, None, D, cu_seqlens_m=cu)
        assert (D == SENTINEL).all(), bad


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("tiles", [True, False])
def test_product_empty_k_and_rows(tile, tiles):
    announce(f"fp8 product empty tile {tile}")
    a, b = gep.fp8_empty(20, 0), gep.fp8_empty(24, 0, tiles=tiles)
    C = torch.randn(20, 24, device="cuda")
    D = torch.full((20, 24), SENTINEL, device="cuda")
    gep.fp8_gemm(a, b, D, C, tile=tile)
    assert torch.equal(D, C)
    gep.fp8_gemm(a, b, D, tile=tile)
    assert (D == 0).all()
    a, b = gep.fp8_empty(0, 64), gep.fp8_empty(24, 64, tiles=tiles)
    assert gep.fp8_gemm(a, b, tile=tile).shape == (0, 24)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("tiles", [True, False])
def test_product_nan_scale(tile, tiles):
    """A NaN block makes the outputs of its row NaN, and only those; one of B those of its columns."""
    announce(f"fp8 product NaN scale tile {tile}")
    x, w = torch.randn(50, 900, device="cuda"), torch.randn(304, 900, device="cuda")
    x[21, 555] = float("nan")
    w[270, 3] = float("inf")
    a, b = gep.fp8_quantize(x), gep.fp8_quantize(w, tiles=tiles)
    D = gep.fp8_gemm(a, b, tile=tile)
    want = torch.zeros(50, 304, dtype=torch.bool, device="cuda")
    want[21] = True
    want[:, 256 if tiles else 270:304 if tiles else 271] = True
    assert torch.equal(D.isnan(), want)


def test_product_in_place_and_stream():
    """C may be D itself; a plan runs on the stream it is given, and repeats bit for bit."""
    announce("fp8 product in place, other stream")
    a, b = gep.fp8_quantize(torch.randn(100, 500, device="cuda")), gep.fp8_quantize(torch.randn(64, 500, device="cuda"), tiles=True)
    C = torch.randn(100, 64, device="cuda")
    want = gep.fp8_gemm(a, b, torch.empty_like(C), C)
    D = C.clone()
    plan = gep.Fp8Plan(a, b, D, D)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan.run(a, b, D, D, stream=s)
    s.synchronize()
    assert torch.equal(D, want)
    with pytest.raises(ValueError):
        plan.run(a, b, D, D.t())
    with pytest.raises(ValueError):
        plan.run(a, gep.fp8_empty(64, 500), D, D)


def test_workspace():
    """A given workspace is used; one that is too small is refused; without one in the C ABI K is
    not split; runs repeat bit for bit."""
    announce("fp8 product workspace")
    import ctypes
    from gemm_epilogue_persistent_amd import _abi
    a, b = gep.fp8_quantize(torch.randn(40, 2048, device="cuda")), gep.fp8_quantize(torch.randn(64, 2048, device="cuda"), tiles=True)
    D, E = torch.empty(40, 64, device="cuda"), torch.empty(40, 64, device="cuda")
    plan = gep.Fp8Plan(a, b, None, D, tile="32", split=4)
    assert plan.workspace_bytes == 4 * 40 * 64 * 4
    plan.run(a, b, None, D)
    ws = torch.full((plan.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")
    plan.run(a, b, None, E, workspace=ws)
    assert torch.equal(D, E)
    with pytest.raises(gep.GemmError):
        plan.run(a, b, None, E, workspace=ws[:-16])
    with pytest.raises(ValueError):
        plan.run(a, b, None, E, workspace=ws.float())
    args = _abi.Fp8GemmArgs(a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(), b.scales.data_ptr(), None,
                            E.data_ptr(), None, None, None, 0)
    E.zero_()
    _abi.check(_abi.load().fp8_gemm_run(plan.handle, ctypes.byref(args), torch.cuda.current_stream().cuda_stream))
    assert torch.equal(E, gep.fp8_gemm(a, b, torch.empty_like(E), tile="32", split=1))


@pytest.mark.parametrize("tile", ["256", "128"])
@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("c,d,post,act", [
    ("bf16", "bf16", None, "none"), ("f16", None, "bf16", "silu"), (None, "bf16", "f16", "gelu_tanh"),
    ("bf16", "f16", "bf16", "silu"), ("f32", "bf16", "bf16", "relu"), (None, "bf16", None, "none")])
def test_product_epilogue_over_tiles(c, d, post, act, tiles, tile):
    """Several tiles a workgroup and edges in both directions: the stores of one tile under the first
    transfers of the next, with each kind of epilogue."""
    announce(f"fp8 product epilogue over tiles c={c} d={d} post={post} {act} tile {tile}")
    n = 5640 if tile == "256" else 2312  # (414 and 608 tiles; a last round of more than half the card is not split)
    run_product(4400 if tile == "256" else 4000, n, 160, tile, tiles, c, d, post, act, seed=41)


@pytest.mark.parametrize("sizes", [None, [1000, 0, 3147, 253]])
def test_product_epilogue_over_deep_tiles(sizes):
    announce(f"fp8 product epilogue over deep tiles {sizes}")
    run_product(4400, 5640, 1000, "256", True, "bf16", "bf16", "bf16", "silu", sizes=sizes, seed=45)


def test_linear_gradients():
    """Both gradients of a linear layer: the products of its quantised operands against the same in 64 bits."""
    announce("fp8 linear gradients")
    m, n, k = 333, 264, 400
    g = torch.Generator().manual_seed(5)
    dy, x, w = (torch.randn(*s, generator=g).bfloat16() for s in ((m, n), (m, k), (n, k)))
    wt = gep.fp8_empty(k, n, tiles=True)
    gep.fp8_quantize(w.cuda(), out_t=wt)
    q, qt, xt = gep.fp8_empty(m, n), gep.fp8_empty(n, m), gep.fp8_empty(k, m)
    gep.fp8_quantize(dy.cuda(), out=q, out_t=qt)
    gep.fp8_quantize(x.cuda(), out_t=xt)
    dx, dw = gep.fp8_gemm(q, wt, torch.empty(m, k, device="cuda")), gep.fp8_gemm(qt, xt, torch.empty(n, k, device="cuda"))
    val = lambda t, tiles=False: R.values(*R.quantize(t.double().numpy(), tiles), t.shape[1], tiles)  # noqa: E731
    for got, a, b in ((dx, val(dy), val(w.t(), True)), (dw, val(dy.t()), val(x.t()))):
        bound = (4 * 4 + 74) * 2.0 ** -24 * (np.abs(a) @ np.abs(b).T) + 128 * 2.0 ** -13 * (largest(a) @ largest(b).T)
        check_product(got, a @ b.T, bound, "f32")


def test_python_refusals():
    a, b = gep.fp8_empty(16, 64), gep.fp8_empty(24, 64, tiles=True)
    D = torch.empty(16, 24, device="cuda")
    g = gep.fp8_empty(24, 64, tiles=True, groups=2)
    cu = torch.tensor([0, 4, 16], dtype=torch.int32, device="cuda")
    for args, kw in (((a, gep.fp8_empty(24, 96), None, D), {}), ((a, g, None, D), {}), ((gep.fp8_empty(16, 64, tiles=True), b, None, D), {}),
                     ((a, b, None, D), dict(cu_seqlens_m=cu)), ((a, g, None, D), dict(cu_seqlens_m=cu[:2])),
                     ((a, g, None, D), dict(cu_seqlens_m=cu.long())), ((a, b, None, D[:8]), {}),
                     ((a, b, None, D), dict(act="tanh")), ((a, b, None, D), dict(tile="512")),
                     ((a, b, None, D.t().contiguous().t()), {})):
        with pytest.raises(ValueError):
            gep.Fp8Plan(*args, **kw)
    with pytest.raises(TypeError):
        gep.Fp8Plan(a, b, None, D.double())
    with pytest.raises(TypeError):
        gep.Fp8Plan(a, D, None, D)
    with pytest.raises(gep.GemmError):
        gep.Fp8Plan(a, b)
    with pytest.raises(gep.GemmError):
        gep.Fp8Plan(a, gep.fp8_empty(20, 64), None, torch.empty(16, 20, device="cuda"))
    x = torch.zeros(16, 64, device="cuda")
    for kw in (dict(out=b), dict(out_t=a), dict(out=a, tiles=True), dict(out=a, out_t=gep.fp8_empty(64, 16, tiles=True)), dict(out=g)):
        with pytest.raises(ValueError):
            gep.fp8_quantize(x, **kw)
    s = gep.fp8_empty(64, 64)
    with pytest.raises(ValueError):
        gep.fp8_quantize(torch.zeros(64, 64, device="cuda"), out=s, out_t=s)
    with pytest.raises(ValueError):
        gep.fp8_quantize(x[:, ::2])
    with pytest.raises(TypeError):
        gep.fp8_quantize(x.double())
    with pytest.raises(TypeError):
        gep.fp8_quantize(x, out=x)
    with pytest.raises(ValueError):
        gep.fp8_dequantize(a, out=torch.empty(16, 63, device="cuda"))
    with pytest.raises(ValueError):
        gep.fp8_dequantize(g)


@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("K", [128, 512, 640, 1536])
def test_nan_stays_in_its_rows(tile, tiles, K):
    """A NaN block of A makes its row NaN and no other, one of B its columns: the scales behind a row's last quad, which are
    another row's, never meet it."""
    announce(f"fp8 product NaN rows {tile} {tiles} {K}")
    A, B = torch.randn(200, K, device="cuda"), torch.randn(264, K, device="cuda")
    A[64:, 0] = float("nan")
    B[128:, K - 1] = float("inf")
    a, b = gep.fp8_quantize(A), gep.fp8_quantize(B, tiles=tiles)
    D = torch.zeros(200, 264, device="cuda")
    gep.Fp8Plan(a, b, None, D, tile=tile, split=1).run(a, b, None, D)
    assert D[:64, :128].isfinite().all() and D[64:].isnan().all() and D[:, 128:].isnan().all()
