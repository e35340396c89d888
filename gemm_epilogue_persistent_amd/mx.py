"""Block-scaled (MX) tensors, their quantiser and their product (binding of
include/mx_mi355x.h; argument checks and marshalling only).

A matrix of e2m1 (4-bit) or e4m3 (8-bit) elements with one power-of-two scale per 32
consecutive values of a row (OCP Microscaling v1.0):

    q = mx_empty(rows, k, "e4m3")                  # storage
    mx_quantize(x, "e4m3", out=q)                  # x (rows, k) in 16 or 32 bits
    mx_quantize(x, "e4m3", out=qt, transpose=True) # the same values as x^T: blocks along columns
    plan = MxPlan(a, b, C, D, PostAct, act="silu") # D = a b^T + C, PostAct = act(that)
    plan.run(a, b, C, D, PostAct)

Grouped: b holds one matrix per expert, (G, n, k), and cu_seqlens_m gives the experts' rows.
"""
import contextlib
import ctypes

import torch

from . import _abi
from ._abi import ACT, DT, MX_FORMAT, MX_TILE

BLOCK = 32
_MOST = (1 << 31) - 1  # sizes of the C ABI are int32
_FLOAT_DT = {torch.float16: DT["f16"], torch.bfloat16: DT["bf16"], torch.float32: DT["f32"]}
_FLOAT_BYTES = {torch.float16: 2, torch.bfloat16: 2, torch.float32: 4}


def _cdiv(a, b):
    return -(-a // b)


# the current stream's pointer by device index (torch.cuda.current_stream builds an object for it,
# which takes as long as a launch)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _allocating(stream):
    """Where a call on `stream` allocates: memory of that stream, so that its first fill and its reuse
    after a free are ordered with the call."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _launch(device, stream, function, *args):
    """function(*args, stream pointer) with `device` current, on `stream` (default: the device's
    current one); raises what it reports."""
    index = device.index
    if index != _current_device():
        with torch.cuda.device(index):
            return _launch(device, stream, function, *args)
    status = function(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if status:
        _abi.check(status)


def _matrix(name, t, dtypes, shape=None, device=None):
    """Checks of a matrix argument on the GPU whose rows are contiguous; its row stride."""
    have = t.shape
    if len(have) != 2 or not t.is_cuda:
        raise ValueError(f"{name}: a matrix on the GPU expected")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if shape is not None and have != shape:
        raise ValueError(f"{name} has shape {tuple(have)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    rows, cols = have
    if rows > _MOST or cols > _MOST:
        raise ValueError(f"{name}: more than 2^31 - 1 rows or columns")
    if rows == 0 or cols == 0:
        return cols
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    if rows == 1:
        return cols
    if ld < cols:
        raise ValueError(f"{name}: rows overlap")
    return ld


class MxTensor:
    """Codes and scales of a (rows, k) MX matrix, or of (G, rows, k) grouped ones.

    codes: uint8, (rows, bytes) or (G, rows, bytes), contiguous; bytes = 32 (e4m3) or 16 (e2m1)
    per block of 32 values, two e2m1 codes to a byte with the even element in the low half; codes
    past k are zero. scales: uint8, (rows / 64, blocks / 16, 64, 16) rounded up (with a leading G
    for grouped ones), contiguous; not 255 past the row's last block. 2^(scale - 127) multiplies
    the block; 255 makes it NaN."""

    __slots__ = ("codes", "scales", "fmt", "k", "rows", "groups", "device")

    def __init__(self, codes, scales, fmt, k):
        if fmt not in MX_FORMAT:
            raise ValueError(f"unknown MX format {fmt!r}")
        k = int(k)
        if k < 0:
            raise ValueError("k must not be negative")
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales are uint8 tensors")
        if codes.dim() not in (2, 3):
            raise ValueError("codes: (rows, bytes) or (G, rows, bytes) expected")
        rows, nb = codes.shape[-2], _cdiv(k, BLOCK)
        lead = tuple(codes.shape[:-2])
        if codes.shape[-1] != nb * (16 if fmt == "e2m1" else 32):
            raise ValueError(f"codes: {codes.shape[-1]} bytes a row do not hold {k} {fmt} values in blocks of 32")
        want = lead + (_cdiv(rows, 64), _cdiv(nb, 16), 64, 16)
        if tuple(scales.shape) != want:
            raise ValueError(f"scales have shape {tuple(scales.shape)}, expected {want}")
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes and scales must be contiguous")
        if codes.device != scales.device:
            raise ValueError("codes and scales are on different devices")
        self.codes, self.scales, self.fmt, self.k = codes, scales, fmt, k
        self.rows, self.groups, self.device = rows, (lead[0] if lead else None), codes.device

    @property
    def shape(self):
        return ((self.groups,) if self.groups is not None else ()) + (self.rows, self.k)

    def group(self, g):
        """The matrix of one group (a view)."""
        if self.groups is None:
            raise ValueError("not a grouped MX tensor")
        return MxTensor(self.codes[g], self.scales[g], self.fmt, self.k)

    def __repr__(self):
        return f"MxTensor({self.fmt}, {tuple(self.shape)}, {self.device})"


def mx_empty(rows, k, fmt, groups=None, device="cuda"):
    """Storage of a (rows, k) MX matrix, or of `groups` of them. The codes are uninitialised; the
    scales start at zero."""
    if fmt not in MX_FORMAT:
        raise ValueError(f"unknown MX format {fmt!r}")
    rows, k = int(rows), int(k)
    if rows < 0 or k < 0 or (groups is not None and groups < 0):
        raise ValueError("negative size")
    lead = () if groups is None else (int(groups),)
    nb = _cdiv(k, BLOCK)
    codes = torch.empty(lead + (rows, nb * (16 if fmt == "e2m1" else 32)), dtype=torch.uint8, device=device)
    scales = torch.zeros(lead + (_cdiv(rows, 64), _cdiv(nb, 16), 64, 16), dtype=torch.uint8, device=device)
    return MxTensor(codes, scales, fmt, k)


def _plain_mx(name, q, device=None):
    if not isinstance(q, MxTensor):
        raise TypeError(f"{name}: an MxTensor expected")
    if q.groups is not None:
        raise ValueError(f"{name}: one matrix expected (see MxTensor.group)")
    if device is not None and q.device != device:
        raise ValueError(f"{name} is on {q.device}, expected {device}")


def mx_quantize(x, fmt, out=None, transpose=False, stream=None):
    """The matrix x (16- or 32-bit floats, rows or columns contiguous) as MX codes: of x with
    blocks along its rows, or (transpose) of x^T with blocks along x's columns. Returns `out`
    (allocated if None). A block that holds a NaN or an infinity becomes NaN (scale 255)."""
    shape = x.shape
    if len(shape) != 2 or not x.is_cuda:
        raise ValueError("x: a matrix on the GPU expected")
    rows, cols = shape
    if transpose:
        shape = (cols, rows)
    if cols > 1 and x.stride(1) != 1 and x.stride(0) == 1:  # columns contiguous: x^T has contiguous rows
        x, rows, cols, transpose = x.t(), cols, rows, not transpose
    ld = _matrix("x", x, _FLOAT_DT)
    if out is None:
        with _allocating(stream):
            out = mx_empty(*shape, fmt, device=x.device)
    else:
        _plain_mx("out", out, x.device)
        if out.fmt != fmt or out.rows != shape[0] or out.k != shape[1]:
            raise ValueError(f"out is {out.fmt} {tuple(out.shape)}, expected {fmt} {tuple(shape)}")
    _launch(x.device, stream, _abi.load().mx_quantize, rows, cols, x.data_ptr(), _FLOAT_DT[x.dtype], ld,
            1 if transpose else 0, MX_FORMAT[fmt], out.codes.data_ptr(), out.scales.data_ptr())
    return out


def mx_dequantize(q, out=None, dtype=torch.bfloat16, stream=None):
    """The values of an MX matrix in `out` (allocated in `dtype` if None), rounded to nearest."""
    _plain_mx("q", q)
    if out is None:
        with _allocating(stream):
            out = torch.empty((q.rows, q.k), dtype=dtype, device=q.device)
    ld = _matrix("out", out, _FLOAT_DT, (q.rows, q.k), q.device)
    _launch(q.device, stream, _abi.load().mx_dequantize, q.rows, q.k, MX_FORMAT[q.fmt], q.codes.data_ptr(),
            q.scales.data_ptr(), out.data_ptr(), _FLOAT_DT[out.dtype], ld)
    return out


def _out(name, t, shape, device):
    if t is None:
        return 0, 0
    ld = _matrix(name, t, _FLOAT_DT, shape, device)
    step = 16 // _FLOAT_BYTES[t.dtype]
    if t.shape[0] <= 1:  # one row: its stride is never used
        ld = _cdiv(ld, step) * step
    return _FLOAT_DT[t.dtype], ld


def _operands(a, b):
    for name, q in (("a", a), ("b", b)):
        if not isinstance(q, MxTensor):
            raise TypeError(f"{name}: an MxTensor expected")


class MxPlan:
    """A validated plan of D = a b^T + C and PostAct = act(a b^T + C) for one problem shape (host
    memory; reusable, from several streams too). a (m, k); b (n, k), or (G, n, k) with
    cu_seqlens_m: int32 of G + 1 row offsets on the GPU, whose values are read by each run. n is a
    multiple of 8. C, D, PostAct: 16- or 32-bit floats, rows contiguous, row strides of whole 16
    bytes; at least one of D, PostAct. tile, split: "auto" and 0, or the kernel to use ("256", "128",
    "32x64", "32", "16x32", "16") and over how many workgroups it shares out a tile's K.

    Sums are held in fp32, but with an e4m3 operand the matrix instruction keeps the products of a block
    of 32 only to 2^-13 of the block's largest: a float32 output is off by about 1e-5 (e2m1 on both sides:
    as an fp32 product).

    Where K is shared out, a run needs a workspace for the partial sums: workspace_bytes of memory that is
    the run's stream's own. The plan keeps one for each stream that it has run on (allocated by the first
    run there, and freed with the plan); a run that is captured into a graph takes one from the graph's
    memory. (Threads that run one plan on one stream at the same time need workspaces of their own.)"""

    def __init__(self, a, b, C=None, D=None, PostAct=None, act="none", cu_seqlens_m=None, tile="auto",
                 split=0):
        self.handle = None
        _operands(a, b)
        _plain_mx("a", a)
        self._sig = self._signature(a, b, C, D, PostAct, cu_seqlens_m)
        if b.device != a.device or not a.codes.is_cuda:
            raise ValueError("a and b must be on one GPU")
        if a.k != b.k:
            raise ValueError("a and b disagree on k")
        grouped = cu_seqlens_m is not None
        if grouped != (b.groups is not None):
            raise ValueError("cu_seqlens_m comes with a grouped b (G, n, k), and only with it")
        if grouped:
            self._check_cu(cu_seqlens_m, b, a.device)
            if b.groups == 0 and a.rows > 0:
                raise ValueError("rows without a group")
        if act not in ACT:
            raise ValueError(f"unknown activation {act!r}")
        if tile not in MX_TILE:
            raise ValueError(f"unknown tile {tile!r}")
        d = _abi.MxGemmDesc()
        d.M, d.N, d.K, d.groups = (_abi.int32(n, v) for n, v in (
            ("rows of a", a.rows), ("rows of b", b.rows), ("k", a.k), ("groups", b.groups or 0)))
        d.a_format, d.b_format = MX_FORMAT[a.fmt], MX_FORMAT[b.fmt]
        shape = (a.rows, b.rows)
        d.c, d.ldc = _out("C", C, shape, a.device)
        d.d, d.ldd = _out("D", D, shape, a.device)
        d.post, d.ldp = _out("PostAct", PostAct, shape, a.device)
        d.act, d.tile, d.split = ACT[act], MX_TILE[tile], _abi.int32("split", split)
        self.desc, self.device = d, a.device
        self._lib = _abi.load()
        h = ctypes.c_void_p()
        _abi.check(self._lib.mx_gemm_create(ctypes.byref(d), ctypes.byref(h)))
        self.handle = h
        n = ctypes.c_int64()
        _abi.check(self._lib.mx_gemm_workspace(h, self._cus(), ctypes.byref(n)))
        self.workspace_bytes = n.value
        self._workspaces, self._workspace = {}, None  # by stream pointer; that of the run before

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            self._lib.mx_gemm_destroy(h)
            self.handle = None

    def _cus(self):
        return torch.cuda.get_device_properties(self.device).multi_processor_count

    @staticmethod
    def _check_cu(cu, b, device):
        if cu.dtype != torch.int32 or cu.device != device or not cu.is_contiguous() or cu.dim() != 1:
            raise ValueError("cu_seqlens_m: contiguous int32 vector on the operands' GPU expected")
        if cu.numel() != b.groups + 1:
            raise ValueError(f"cu_seqlens_m: {b.groups + 1} offsets expected")

    @staticmethod
    def _signature(a, b, C, D, PostAct, cu):
        return (a.fmt, a.codes.shape, a.k, a.device, b.fmt, b.codes.shape, b.device) + tuple(
            None if t is None else (t.dtype, t.shape, t.stride(), t.device) for t in (C, D, PostAct, cu))

    def run(self, a, b, C=None, D=None, PostAct=None, cu_seqlens_m=None, stream=None, workspace=None):
        """Enqueue on `stream` (default: torch's current stream of the operands' device). The
        tensors are laid out as those the plan was made for. workspace: instead of the plan's own, a
        uint8 tensor of plan.workspace_bytes that nothing else uses meanwhile."""
        if self._signature(a, b, C, D, PostAct, cu_seqlens_m) != self._sig:
            raise ValueError("the operands are not laid out as those this plan was made for")
        if workspace is None:
            if self.workspace_bytes:
                workspace = self._stream_workspace(stream)
        elif workspace.device != self.device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace: contiguous uint8 tensor on the operands' GPU expected")
        args = _abi.MX_GEMM_ARGS.pack(a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(), b.scales.data_ptr(),
                                      *[0 if t is None else t.data_ptr() for t in (C, D, PostAct, cu_seqlens_m, workspace)],
                                      0 if workspace is None else workspace.numel())
        _launch(self.device, stream, self._lib.mx_gemm_run, self.handle, args)

    def _stream_workspace(self, stream):
        """The workspace of a run on `stream`. It is allocated on that very stream: a block that the
        allocator hands out on another one may still be in use by what was enqueued there before."""
        if self.device.index != _current_device():
            with torch.cuda.device(self.device):
                return self._stream_workspace(stream)
        with _allocating(stream):
            if torch.cuda.is_current_stream_capturing():  # (not kept: a later graph may outlive this one)
                return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)
            raw = _raw_stream(self.device.index)
            workspace = self._workspaces.get(raw)
            if workspace is None:
                workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)
                self._workspaces[raw] = workspace
        self._workspace = workspace
        return workspace

    def tile(self, num_cus=None):
        """(kernel, split) this plan runs with on a device with num_cus compute units."""
        t, n = ctypes.c_int32(), ctypes.c_int32()
        _abi.check(self._lib.mx_gemm_plan_tile(self.handle, _abi.int32("num_cus", num_cus or self._cus()), ctypes.byref(t), ctypes.byref(n)))
        return next(k for k, v in MX_TILE.items() if v == t.value), n.value


def mx_gemm(a, b, D=None, C=None, PostAct=None, act="none", cu_seqlens_m=None, stream=None, tile="auto",
            split=0):
    """One-shot product: plan and enqueue. Without D and PostAct, D is allocated in bf16. Returns
    D, or PostAct without D."""
    _operands(a, b)
    with _allocating(stream):
        if D is None and PostAct is None:
            D = torch.empty((a.rows, b.rows), dtype=torch.bfloat16, device=a.device)
        plan = MxPlan(a, b, C, D, PostAct, act, cu_seqlens_m, tile, split)
    plan.run(a, b, C, D, PostAct, cu_seqlens_m, stream)
    return D if D is not None else PostAct
