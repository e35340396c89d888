"""Fused RMS norm with residual addition and MX output, and its gradients (binding of
include/mx_mi355x.h; argument checks and marshalling only).

    h = x + residual (rounded to x's type)    rstd = 1 / sqrt(mean(h^2) + eps)
    y = h * rstd * weight, in x's type and / or as an MX matrix
"""
import torch

from . import _abi
from ._abi import MX_FORMAT
from .mx import _FLOAT_DT, _allocating, _launch, _matrix, _plain_mx


def _vector(name, t, n, dtype, device):
    if t.shape != (n,) or t.dtype != dtype or t.device != device or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name}: contiguous {dtype} vector of {n} on {device} expected")
    return t.data_ptr()


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def rmsnorm(x, weight, residual=None, eps=1e-5, h=None, y=None, q=None, rstd=None, stream=None):
    """RMS norm over the rows of x (rows, cols), 16- or 32-bit floats with contiguous rows.

    h: where x + residual goes (may be x or residual itself; only with a residual; without h the
    sum is not kept). y: the norm in x's type; q: an MxTensor (rows, cols) quantised from the
    unrounded norm; without either, y is allocated. rstd: float32 (rows,), what rmsnorm_backward
    takes. Returns y, or q without y."""
    types = (x.dtype,)
    if x.dtype not in _FLOAT_DT:
        raise TypeError(f"x: unsupported dtype {x.dtype}")
    ldx = _matrix("x", x, types)
    dev, shape = x.device, x.shape
    rows, cols = shape
    if y is None and q is None:
        with _allocating(stream):
            y = torch.empty(shape, dtype=x.dtype, device=dev)
    if h is not None and residual is None:
        raise ValueError("h without a residual (it would be x)")
    if q is not None:
        _plain_mx("q", q, dev)
        if q.rows != rows or q.k != cols:
            raise ValueError(f"q has shape {tuple(q.shape)}, expected {tuple(shape)}")
    a = _abi.RMSNORM_ARGS.pack(
        rows, cols, _FLOAT_DT[x.dtype], MX_FORMAT[q.fmt] if q is not None else 0, eps,
        x.data_ptr(), _ptr(residual), _vector("weight", weight, cols, x.dtype, dev), _ptr(h), _ptr(y),
        q.codes.data_ptr() if q is not None else 0, q.scales.data_ptr() if q is not None else 0,
        _vector("rstd", rstd, rows, torch.float32, dev) if rstd is not None else 0,
        ldx, _matrix("residual", residual, types, shape, dev) if residual is not None else 0,
        _matrix("h", h, types, shape, dev) if h is not None else 0,
        _matrix("y", y, types, shape, dev) if y is not None else 0)
    _launch(dev, stream, _abi.load().rmsnorm_forward, a)
    return y if y is not None else q


def rmsnorm_backward_workspace(rows, cols):
    """Bytes of device memory that rmsnorm_backward takes as its workspace."""
    n = _abi.load().rmsnorm_backward_workspace(_abi.int32("rows", rows), _abi.int32("cols", cols))
    if n < 0:
        raise ValueError("negative size, or more than 2^30 rows or 2^24 columns")
    return n


def rmsnorm_backward(dy, h, weight, rstd, dx=None, dw=None, dres=None, workspace=None, stream=None):
    """Gradients of rmsnorm from dy (the gradient of y), the h and rstd it kept and, if given, dres
    (the gradient that reaches h past the norm). dx: with respect to h, hence to x and to the
    residual (may be dy or dres itself); dw: float32 (cols,). workspace: a uint8 tensor of
    rmsnorm_backward_workspace(rows, cols) bytes. What is None is allocated. Returns (dx, dw)."""
    if h.dtype not in _FLOAT_DT:
        raise TypeError(f"h: unsupported dtype {h.dtype}")
    types = (h.dtype,)
    ldh = _matrix("h", h, types)
    dev, shape = h.device, h.shape
    rows, cols = shape
    if dx is None or dw is None or workspace is None:
        with _allocating(stream):
            if dx is None:
                dx = torch.empty(shape, dtype=h.dtype, device=dev)
            if dw is None:
                dw = torch.empty(cols, dtype=torch.float32, device=dev)
            if workspace is None:
                workspace = torch.empty(rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)
    if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: contiguous uint8 tensor on the operands' GPU expected")
    a = _abi.RMSNORM_BACKWARD_ARGS.pack(
        rows, cols, _FLOAT_DT[h.dtype], dy.data_ptr(), h.data_ptr(), _vector("weight", weight, cols, h.dtype, dev),
        _vector("rstd", rstd, rows, torch.float32, dev), _ptr(dres), dx.data_ptr(),
        _vector("dw", dw, cols, torch.float32, dev), workspace.data_ptr(), workspace.numel(),
        _matrix("dy", dy, types, shape, dev), ldh,
        _matrix("dres", dres, types, shape, dev) if dres is not None else 0, _matrix("dx", dx, types, shape, dev))
    _launch(dev, stream, _abi.load().rmsnorm_backward, a)
    return dx, dw
