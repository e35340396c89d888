"""Plain 64-bit implementation of the 8-bit matrices with a scale per 128 values (numpy, CPU), written from the
format's definition."""
import numpy as np

BLOCK = 128


def magnitudes():
    return np.array([i * 2.0 ** -9 for i in range(8)] + [(8 + i) * 2.0 ** (e - 3) for e in range(-6, 9) for i in range(8)])[:127]


def factor(top):
    """r of blocks of largest magnitude `top` (float64): 448 / top in fp32, at most 2^126, cut to 13 bits."""
    with np.errstate(divide="ignore", over="ignore"):
        r = np.minimum((448.0 / top).astype(np.float32), np.float32(2.0 ** 126))
    m, e = np.frexp(r.astype(np.float64))
    return np.ldexp(np.floor(np.ldexp(m, 13)), e - 13)


def round_code(v):
    """Codes of values within +-448, nearest, ties to even."""
    m = magnitudes()
    between = (m[1:] + m[:-1]) / 2
    lo, hi = np.searchsorted(between, np.abs(v), side="left"), np.searchsorted(between, np.abs(v), side="right")
    code = np.where(lo == hi, lo, lo + lo % 2)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantize(x, tiles=False):
    """(codes (rows, 16-byte rows), scales (rows or row tiles, blocks)) of x (rows, k) in float64; NaN scales of
    blocks that are not finite."""
    rows, k = x.shape
    tall = BLOCK if tiles else 1
    nb, nt = -(-k // BLOCK), -(-rows // tall)
    b = np.zeros((nt * tall, nb * BLOCK))
    b[:rows, :k] = x
    b = b.reshape(nt, tall, nb, BLOCK)
    bad = ~np.isfinite(b).all((1, 3))
    top = np.abs(np.where(np.isfinite(b), b, 0)).max((1, 3))
    r = factor(top)
    with np.errstate(invalid="ignore"):
        v = np.clip(np.where(bad[:, None, :, None], 0.0, b * r[:, None, :, None]), -448, 448)
    codes = np.where(bad[:, None, :, None], 0, round_code(v)).reshape(nt * tall, nb * BLOCK)[:rows]
    out = np.zeros((rows, -(-k // 16) * 16), np.uint8)
    out[:, :k] = codes[:, :k]
    scales = np.where(bad, np.nan, (1.0 / r)).astype(np.float32)
    return out, scales


def spread(scales, rows, k, tiles):
    """The scale of every value (rows, k)."""
    s = scales.astype(np.float64)
    s = np.repeat(s, BLOCK, 0)[:rows] if tiles else s
    return np.repeat(s, BLOCK, 1)[:, :k]


def values(codes, scales, k, tiles=False):
    m = magnitudes()
    c = codes[:, :k]
    v = np.where(c & 128, -1.0, 1.0) * np.append(m, np.nan)[c & 127]
    return v * spread(scales, codes.shape[0], k, tiles)


def store_scales(scales, tiles=False, fill=0.0):
    """The storage order; `fill` in the rows past the end, zeros past the last block."""
    rows, nb = scales.shape
    nq = -(-nb // 4)
    if tiles:
        out = np.zeros((rows, nq * 4), np.float32)
        out[:, :nb] = scales
        return out
    out = np.full((-(-rows // 64) * 64, nq * 4), fill, np.float32)
    out[:rows] = 0
    out[:rows, :nb] = scales
    return np.ascontiguousarray(out.reshape(-1, 64, nq, 4).transpose(0, 2, 1, 3))


def load_scales(stored, rows, tiles=False):
    """(rows or row tiles, whole quads of blocks)."""
    if tiles:
        return stored
    t, nq = stored.shape[:2]
    return stored.transpose(0, 2, 1, 3).reshape(t * 64, nq * 4)[:rows]


def act(x, name):
    if name == "relu":
        return np.where(x > 0, x, 0.0)
    if name == "relu_sq":
        return np.where(x > 0, x, 0.0) ** 2
    if name in ("gelu_tanh", "silu"):
        z = x if name == "silu" else 2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
        with np.errstate(over="ignore"):
            return x / (1 + np.exp(-z))
    return x


def slope(x, name):
    if name == "relu":
        return (x > 0).astype(float)
    if name == "relu_sq":
        return 2 * np.where(x > 0, x, 0.0)
    if name in ("gelu_tanh", "silu"):
        c = 2 * np.sqrt(2 / np.pi)
        z, dz = (x, 1.0) if name == "silu" else (c * (x + 0.044715 * x ** 3), c * (1 + 3 * 0.044715 * x * x))
        with np.errstate(over="ignore"):
            s, rest = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
        return s + x * s * rest * dz
    return np.ones_like(x)
