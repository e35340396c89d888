"""Plain 64-bit implementation (numpy) of the MX format, its product and the RMS norm, for the
tests. Shares nothing with the library.

e2m1: 1 sign, 2 exponent, 1 fraction bits, largest 6 (emax 2); e4m3: 1, 4, 3, largest 448 (emax
8). A block of 32 values has scale byte s = 127 + floor(log2 max) - emax in [0, 254]; 255 is NaN.
"""
import numpy as np

EMAX = {"e2m1": 2, "e4m3": 8}
ROW_BYTES = {"e2m1": 16, "e4m3": 32}  # of a block


def magnitudes(fmt):
    """Code -> magnitude, ascending."""
    out = []
    frac, bias, n = (1, 1, 8) if fmt == "e2m1" else (3, 7, 127)
    for c in range(n):
        e, f = c >> frac, c & ((1 << frac) - 1)
        out.append(f * 2.0 ** (1 - bias - frac) if e == 0 else (1 + f / 2.0 ** frac) * 2.0 ** (e - bias))
    return np.array(out)


def round_code(a, fmt):
    """Codes of magnitudes a (64-bit, scaled): nearest, ties to the even code, saturated."""
    m = magnitudes(fmt)
    hi = np.clip(np.searchsorted(m, a, side="left"), 0, len(m) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - m[lo], m[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(a >= m[-1], len(m) - 1, np.where(up, hi, lo))


def blocks(x):
    rows, k = x.shape
    nb = -(-k // 32)
    out = np.zeros((rows, nb * 32), dtype=np.float64)
    out[:, :k] = x
    return out.reshape(rows, nb, 32)


def scale_bytes(x, fmt):
    """(rows, blocks) of the scale bytes of x (rows, k)."""
    b = np.abs(blocks(x))
    bad = ~np.isfinite(b).all(-1)
    a = np.where(np.isfinite(b), b, 0).max(-1)
    _, e = np.frexp(a)  # a = f 2^e, f in [1/2, 1)
    s = np.where(a > 0, np.clip(127 + e - 1 - EMAX[fmt], 0, 254), 0)
    return np.where(bad, 255, s).astype(np.int64)


def quantize(x, fmt):
    """Element codes (rows, blocks * 32) with the sign bit, and scale bytes (rows, blocks)."""
    s = scale_bytes(x, fmt)
    b = blocks(x)
    ok = (s != 255)[..., None]
    v = np.where(ok, b, 0.0) / 2.0 ** (s[..., None] - 127.0)
    c = round_code(np.abs(v), fmt)
    sign = np.signbit(v) & ok
    c = c | (sign.astype(np.int64) << (3 if fmt == "e2m1" else 7))
    return c.reshape(x.shape[0], -1), s


def values(codes, s, fmt, k):
    """The 64-bit values of element codes and scale bytes."""
    top = 8 if fmt == "e2m1" else 128
    m = magnitudes(fmt)
    mag = np.where((codes & (top - 1)) < len(m), m[np.minimum(codes & (top - 1), len(m) - 1)], np.nan)
    v = np.where(codes & top, -mag, mag).reshape(codes.shape[0], -1, 32)
    sc = np.where(s == 255, np.nan, 2.0 ** (s - 127.0))
    return (v * sc[..., None]).reshape(codes.shape[0], -1)[:, :k]


def pack(codes, fmt):
    """Element codes as stored bytes."""
    c = codes.astype(np.uint8)
    return c if fmt == "e4m3" else (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def unpack(stored, fmt):
    s = stored.astype(np.int64)
    if fmt == "e4m3":
        return s
    return np.stack([s & 15, s >> 4], -1).reshape(s.shape[0], -1)


def store_scales(s, fill=0):
    """Scale bytes (rows, blocks) in storage order; rows and blocks past the end hold `fill`."""
    rows, nb = s.shape
    out = np.full((-(-rows // 64) * 64, -(-nb // 16) * 16), fill, dtype=np.uint8)
    out[:rows, nb:] = 0
    out[:rows, :nb] = s
    return np.ascontiguousarray(out.reshape(out.shape[0] // 64, 64, -1, 16).transpose(0, 2, 1, 3))


def load_scales(t, rows):
    """Storage order -> (rows, padded blocks)."""
    return t.transpose(0, 2, 1, 3).reshape(t.shape[0] * 64, -1)[:rows].astype(np.int64)


def act(x, name):
    if name == "relu":
        return np.maximum(x, 0)
    if name == "relu_sq":
        return np.maximum(x, 0) ** 2
    if name == "gelu_tanh":
        return 0.5 * x * (1 + np.tanh(np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)))
    if name == "silu":
        with np.errstate(over="ignore"):
            return x / (1 + np.exp(-x))
    return x
