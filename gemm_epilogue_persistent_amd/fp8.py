"""8-bit matrices with a scale per 128 values, their quantiser and product, and activations that keep their input in 8
bits for the backward pass (binding of include/fp8_mi355x.h; argument checks and marshalling only).

A matrix of e4m3 elements with one fp32 scale per 128 consecutive values of a row (activations, gradients)
or per tile of 128 rows by 128 values (weights):

    w = fp8_quantize(weight, tiles=True)              # (n, k), laid out once
    q = fp8_empty(rows, k)                            # storage
    fp8_quantize(x, out=q)                            # x (rows, k) in 16 or 32 bits
    fp8_quantize(x, out=q, out_t=qt)                  # and x^T, with blocks along x's columns, in the same pass
    plan = Fp8Plan(a, b, C, D, PostAct, act="silu")   # D = a b^T + C, PostAct = act(that)
    plan.run(a, b, C, D, PostAct)
    fp8_act(x, "silu", saved=kept, q=q)               # q = act(x) for the next product, x itself kept in 8 bits
    fp8_act_backward(dy, kept, "silu", q=dq, qt=dqt)  # dy act'(x) from them, for both products of the backward pass

Grouped: b holds one matrix per expert, (G, n, k), and cu_seqlens_m gives the experts' rows.
"""
import ctypes

import torch

from . import _abi
from ._abi import ACT, FP8_TILE
from .mx import _FLOAT_DT, _allocating, _cdiv, _launch, _matrix, _out, _PlanBase

BLOCK = 128
_ROWS, _TILES = 0, 1


def _scale_shape(rows, k, tiles):
    quads = _cdiv(_cdiv(k, BLOCK), 4)
    return (_cdiv(rows, BLOCK), quads * 4) if tiles else (_cdiv(rows, 64), quads, 64, 4)


class Fp8Tensor:
    """Codes and scales of a (rows, k) matrix, or of (G, rows, k) grouped ones.

    codes: uint8 (e4m3), (rows, bytes) or (G, rows, bytes), contiguous; bytes = k rounded up to 16, the codes
    past k zero. scales: float32, contiguous; a scale per 128 values of a row: (rows / 64, blocks / 4, 64, 4)
    rounded up; per tile of 128 x 128 (tiles): (rows / 128, blocks rounded up to a multiple of 4). Each with a
    leading G for grouped ones; below 2^63 past the row's last block. A value is code * scale; a NaN scale
    makes its block NaN."""

    __slots__ = ("codes", "scales", "k", "rows", "groups", "tiles", "device")

    def __init__(self, codes, scales, k):
        k = int(k)
        if k < 0:
            raise ValueError("k must not be negative")
        if codes.dtype != torch.uint8 or scales.dtype != torch.float32:
            raise TypeError("codes are a uint8 tensor and scales a float32 one")
        if codes.dim() not in (2, 3):
            raise ValueError("codes: (rows, bytes) or (G, rows, bytes) expected")
        rows, lead = codes.shape[-2], tuple(codes.shape[:-2])
        if codes.shape[-1] != _cdiv(k, 16) * 16:
            raise ValueError(f"codes: rows of {_cdiv(k, 16) * 16} bytes expected for {k} values, not {codes.shape[-1]}")
        tiles = scales.dim() == codes.dim()
        want = lead + _scale_shape(rows, k, tiles)
        if tuple(scales.shape) != want:
            raise ValueError(f"scales have shape {tuple(scales.shape)}, expected {lead + _scale_shape(rows, k, False)} "
                             f"or, of tiles, {lead + _scale_shape(rows, k, True)}")
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes and scales must be contiguous")
        if codes.device != scales.device:
            raise ValueError("codes and scales are on different devices")
        self.codes, self.scales, self.k, self.tiles = codes, scales, k, tiles
        self.rows, self.groups, self.device = rows, (lead[0] if lead else None), codes.device

    @property
    def shape(self):
        return ((self.groups,) if self.groups is not None else ()) + (self.rows, self.k)

    def group(self, g):
        """The matrix of one group (a view)."""
        if self.groups is None:
            raise ValueError("not a grouped FP8 tensor")
        return Fp8Tensor(self.codes[g], self.scales[g], self.k)

    def __repr__(self):
        return f"Fp8Tensor({tuple(self.shape)}, {'tiles' if self.tiles else 'rows'}, {self.device})"


def fp8_empty(rows, k, tiles=False, groups=None, device="cuda"):
    """Storage of a (rows, k) FP8 matrix, or of `groups` of them, with a scale per 128 values of a row or
    (tiles) per 128 x 128. The codes are uninitialised; the scales start at zero."""
    rows, k = int(rows), int(k)
    if rows < 0 or k < 0 or (groups is not None and groups < 0):
        raise ValueError("negative size")
    lead = () if groups is None else (int(groups),)
    codes = torch.empty(lead + (rows, _cdiv(k, 16) * 16), dtype=torch.uint8, device=device)
    return Fp8Tensor(codes, torch.zeros(lead + _scale_shape(rows, k, bool(tiles)), dtype=torch.float32, device=device), k)


def _plain(name, q, shape=None, device=None, tiles=None):
    """Checks of one FP8 matrix; the addresses of its codes and scales (0, 0 for None)."""
    if q is None:
        return 0, 0
    if not isinstance(q, Fp8Tensor):
        raise TypeError(f"{name}: an Fp8Tensor expected")
    if q.groups is not None:
        raise ValueError(f"{name}: one matrix expected (see Fp8Tensor.group)")
    if not q.codes.is_cuda:
        raise ValueError(f"{name}: a matrix on the GPU expected")
    if device is not None and q.device != device:
        raise ValueError(f"{name} is on {q.device}, expected {device}")
    if shape is not None and (q.rows, q.k) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(q.shape)}, expected {tuple(shape)}")
    if tiles is not None and q.tiles != tiles:
        raise ValueError(f"{name}: a scale per {'128 x 128 tile' if tiles else '128 values of a row'} expected")
    return q.codes.data_ptr(), q.scales.data_ptr()


def fp8_quantize(x, out=None, out_t=None, tiles=None, stream=None):
    """The matrix x (16- or 32-bit floats, rows or columns contiguous) as an FP8 one, in `out`, and that of x^T in
    `out_t` (blocks along x's columns, or the same tiles), in one pass over x. Without either, `out` is
    allocated, with a scale per 128 values of a row or (tiles) per 128 x 128; given ones say themselves which.
    Returns out, or out_t without out. A block that holds a NaN or an infinity becomes NaN."""
    shape = x.shape
    if len(shape) != 2 or not x.is_cuda:
        raise ValueError("x: a matrix on the GPU expected")
    rows, cols = shape
    given = out if out is not None else out_t
    if given is None:
        with _allocating(stream):
            given = out = fp8_empty(rows, cols, tiles=bool(tiles), device=x.device)
    if not isinstance(given, Fp8Tensor):
        raise TypeError("out: an Fp8Tensor expected")
    if tiles is None:
        tiles = given.tiles
    q = _plain("out", out, (rows, cols), x.device, tiles)
    qt = _plain("out_t", out_t, (cols, rows), x.device, tiles)
    if q[0] and q[0] == qt[0]:
        raise ValueError("out and out_t are one matrix")
    if cols > 1 and x.stride(1) != 1 and x.stride(0) == 1:  # columns contiguous: x^T has contiguous rows
        x, rows, cols, q, qt = x.t(), cols, rows, qt, q
    ld = _matrix("x", x, _FLOAT_DT)
    _launch(x.device, stream, _abi.load().fp8_quantize, rows, cols, x.data_ptr(), _FLOAT_DT[x.dtype], ld,
            _TILES if tiles else _ROWS, *q, *qt)
    return out if out is not None else out_t


def fp8_dequantize(q, out=None, dtype=torch.bfloat16, stream=None):
    """The values of an FP8 matrix in `out` (allocated in `dtype` if None), rounded to nearest."""
    codes, scales = _plain("q", q)
    if q is None:
        raise TypeError("q: an Fp8Tensor expected")
    if out is None:
        with _allocating(stream):
            out = torch.empty((q.rows, q.k), dtype=dtype, device=q.device)
    ld = _matrix("out", out, _FLOAT_DT, (q.rows, q.k), q.device)
    _launch(q.device, stream, _abi.load().fp8_dequantize, _abi.int32("rows", q.rows), _abi.int32("k", q.k),
            _TILES if q.tiles else _ROWS, codes, scales, out.data_ptr(), _FLOAT_DT[out.dtype], ld)
    return out


def _activation(act):
    if act not in ACT:
        raise ValueError(f"unknown activation {act!r}")
    return ACT[act]


def fp8_act(x, act, saved=None, q=None, y=None, stream=None):
    """An activation between two products, in one pass over x (rows, cols; 16- or 32-bit floats, rows
    contiguous): saved: x itself in 8 bits, for fp8_act_backward; q: act(x) in 8 bits, for the next product; y: act(x)
    in x's type (may be x itself). Those not wanted are None; without any, y is allocated. Both FP8
    matrices have a scale per 128 values of a row. Returns y, or q without y, or saved without both."""
    types = (x.dtype,)
    if x.dtype not in _FLOAT_DT:
        raise TypeError(f"x: unsupported dtype {x.dtype}")
    code = _activation(act)
    ldx = _matrix("x", x, types)
    dev, shape = x.device, x.shape
    if saved is None and q is None and y is None:
        with _allocating(stream):
            y = torch.empty(shape, dtype=x.dtype, device=dev)
    kept, nxt = _plain("saved", saved, shape, dev, False), _plain("q", q, shape, dev, False)
    if kept[0] and kept[0] == nxt[0]:
        raise ValueError("saved and q are one matrix")
    ldy = _matrix("y", y, types, shape, dev) if y is not None else 0
    a = _abi.FP8_ACT_ARGS.pack(*shape, _FLOAT_DT[x.dtype], code, x.data_ptr(), *kept, *nxt,
                               y.data_ptr() if y is not None else 0, ldx, ldy)
    _launch(dev, stream, _abi.load().fp8_act_forward, a)
    return y if y is not None else q if q is not None else saved


def fp8_act_backward(dy, saved, act, dx=None, q=None, qt=None, y=None, yt=None, stream=None):
    """The backward pass of fp8_act from what it saved, in one pass over dy and the 8 bits. With x^ the values of `saved`:

      dx = dy act'(x^), in dy's type (dx; may be dy itself), in 8 bits (q) and in 8 bits transposed (qt, blocks
      along the rows of dy: the operand of the weight's gradient)
      y = act(x^), in 16 or 32 bits (y), and in 8 bits transposed (yt: the operand of the gradient of the
      weight behind the activation)

    Those not wanted are None, but not all of them; dy is None without dx, q and qt. (act "none" with yt alone
    turns a checkpoint's blocks to the other axis.) Returns nothing."""
    _plain("saved", saved, tiles=False)
    if saved is None:
        raise TypeError("saved: an Fp8Tensor expected")
    dev, shape = saved.device, (saved.rows, saved.k)
    code = _activation(act)
    wide = [t for t in (dy, dx, y) if t is not None]
    dtype = wide[0].dtype if wide else torch.bfloat16
    if dtype not in _FLOAT_DT:
        raise TypeError(f"unsupported dtype {dtype}")
    if (dy is not None) != (dx is not None or q is not None or qt is not None):
        raise ValueError("dy comes with dx, q or qt")
    if dy is None and y is None and yt is None:
        raise ValueError("no output")
    lds = [_matrix(n, t, (dtype,), shape, dev) if t is not None else 0 for n, t in (("dy", dy), ("dx", dx), ("y", y))]
    ptr = lambda t: t.data_ptr() if t is not None else 0  # noqa: E731
    back = (saved.k, saved.rows)
    a = _abi.FP8_ACT_BACKWARD_ARGS.pack(
        _abi.int32("rows", saved.rows), _abi.int32("cols", saved.k), _FLOAT_DT[dtype], code, ptr(dy),
        saved.codes.data_ptr(), saved.scales.data_ptr(), ptr(dx), *_plain("q", q, shape, dev, False),
        *_plain("qt", qt, back, dev, False), ptr(y), *_plain("yt", yt, back, dev, False), *lds)
    _launch(dev, stream, _abi.load().fp8_act_backward, a)


def _operands(a, b):
    for name, q in (("a", a), ("b", b)):
        if not isinstance(q, Fp8Tensor):
            raise TypeError(f"{name}: an Fp8Tensor expected")


class Fp8Plan(_PlanBase):
    """A validated plan of D = a b^T + C and PostAct = act(a b^T + C) for one problem shape (host memory;
    reusable, from several streams too). a (m, k) with a scale per 128 values of a row; b (n, k), or (G, n, k) with
    cu_seqlens_m: int32 of G + 1 row offsets on the GPU, whose values are read by each run; b's scales are of
    tiles (weights) or of rows (the gradient of a weight: a = dY^T, b = X^T, blocks along the tokens).
    n is a multiple of 8. C, D, PostAct: 16- or 32-bit floats, rows contiguous, row strides of whole 16
    bytes; at least one of D, PostAct. tile, split: "auto" and 0, or the kernel to use ("256", "128",
    "64", "32", "16x32", "16") and over how many workgroups it shares out a tile's K.

    The matrix instruction sums a block's 128 products (each kept to 2^-13 of the largest of 32), and blocks are
    scaled and added in fp32: a float32 output is off by about 1e-5.

    Where K is shared out, a run needs a workspace for the partial sums: workspace_bytes of memory that is
    the run's stream's own. The plan keeps one for each stream that it has run on (allocated by the first
    run there, and freed with the plan); a run that is captured into a graph takes one from the graph's
    memory. (Threads that run one plan on one stream at the same time need workspaces of their own.)"""

    _create, _destroy, _run, _plan_tile, _workspace_size = (
        "fp8_gemm_create", "fp8_gemm_destroy", "fp8_gemm_run", "fp8_gemm_plan_tile", "fp8_gemm_workspace")
    _tiles = FP8_TILE

    def __init__(self, a, b, C=None, D=None, PostAct=None, act="none", cu_seqlens_m=None, tile="auto", split=0):
        self.handle = None
        _operands(a, b)
        _plain("a", a, tiles=False)
        self._check_operands(a, b, cu_seqlens_m, act, tile)
        d = _abi.Fp8GemmDesc()
        d.M, d.N, d.K, d.groups = (_abi.int32(n, v) for n, v in (
            ("rows of a", a.rows), ("rows of b", b.rows), ("k", a.k), ("groups", b.groups or 0)))
        d.b_scaling = _TILES if b.tiles else _ROWS
        self._finish(d, a, b, C, D, PostAct, act, cu_seqlens_m, tile, split)

    @staticmethod
    def _signature(a, b, C, D, PostAct, cu):
        return (a.codes.shape, a.k, a.tiles, a.device, b.codes.shape, b.tiles, b.device) + tuple(
            None if t is None else (t.dtype, t.shape, t.stride(), t.device) for t in (C, D, PostAct, cu))


def fp8_gemm(a, b, D=None, C=None, PostAct=None, act="none", cu_seqlens_m=None, stream=None, tile="auto", split=0):
    """One-shot product: plan and enqueue. Without D and PostAct, D is allocated in bf16. Returns D, or
    PostAct without D."""
    _operands(a, b)
    with _allocating(stream):
        if D is None and PostAct is None:
            D = torch.empty((a.rows, b.rows), dtype=torch.bfloat16, device=a.device)
        plan = Fp8Plan(a, b, C, D, PostAct, act, cu_seqlens_m, tile, split)
    plan.run(a, b, C, D, PostAct, cu_seqlens_m, stream)
    return D if D is not None else PostAct
