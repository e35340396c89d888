"""CPU tests of the MX and RMS norm entry points: exports, sizes, and every refusal, all of them
before any HIP call (fake pointers, no GPU)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import gemm_epilogue_persistent_amd as gep
import mx_ref as R
from gemm_epilogue_persistent_amd import _abi

P = 4096  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        from gemm_epilogue_persistent_amd import build
        build.build()
    return _abi.load()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(_abi.MX_HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b((?:mx|rmsnorm)_[a-z_]+)\s*\(", text))
    assert {"mx_quantize", "mx_dequantize", "mx_gemm_create", "mx_gemm_run", "rmsnorm_forward",
            "rmsnorm_backward"} <= names
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("rows,k", [(0, 0), (1, 1), (3, 32), (64, 512), (65, 513), (100, 1000)])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_storage_sizes(lib, rows, k, fmt):
    nb = -(-k // 32)
    assert lib.mx_code_bytes(rows, k, _abi.MX_FORMAT[fmt]) == rows * nb * R.ROW_BYTES[fmt]
    assert lib.mx_scale_bytes(rows, k) == -(-rows // 64) * -(-nb // 16) * 1024
    q = gep.mx_empty(rows, k, fmt, device="cpu")
    assert q.codes.numel() == lib.mx_code_bytes(rows, k, _abi.MX_FORMAT[fmt])
    assert q.scales.numel() == lib.mx_scale_bytes(rows, k) and not q.scales.any()
    assert q.shape == (rows, k)
    g = gep.mx_empty(rows, k, fmt, groups=3, device="cpu")
    assert g.shape == (3, rows, k) and g.group(1).shape == (rows, k)
    assert lib.mx_code_bytes(-1, 1, 0) == -1 and lib.mx_code_bytes(1, 1, 2) == -1 and lib.mx_scale_bytes(1, -1) == -1


def test_reference_tables():
    assert R.magnitudes("e2m1").tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    m = R.magnitudes("e4m3")
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(m, t)
    # ties go to the even code, larger values to the largest
    assert R.round_code(np.array([0.25, 0.75, 1.25, 2.5, 5.0, 9.0]), "e2m1").tolist() == [0, 2, 2, 4, 6, 7]


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), _abi.INVALID_ARG), (dict(cols=-1), _abi.INVALID_ARG), (dict(rows=(1 << 30) + 1), _abi.UNSUPPORTED),
    (dict(x=None), _abi.INVALID_ARG), (dict(x=P + 1), _abi.ALIGNMENT), (dict(dt=4), _abi.INVALID_ARG),
    (dict(dt=0), _abi.INVALID_ARG), (dict(ld=31), _abi.INVALID_ARG), (dict(ld=-1), _abi.INVALID_ARG),
    (dict(rows=1, ld=-1), _abi.UNSUPPORTED), (dict(ld=(1 << 48) + 1), _abi.UNSUPPORTED), (dict(tr=2), _abi.INVALID_ARG),
    (dict(fmt=2), _abi.INVALID_ARG), (dict(codes=None), _abi.INVALID_ARG), (dict(codes=P + 8), _abi.ALIGNMENT),
    (dict(scales=None), _abi.INVALID_ARG),
])
def test_quantize_refusals(lib, kw, status):
    a = dict(rows=4, cols=32, x=P, dt=_abi.DT["bf16"], ld=32, tr=0, fmt=1, codes=P, scales=P)
    a.update(kw)
    assert lib.mx_quantize(*a.values(), None) == status and lib.gemm_last_error()
    if "tr" not in kw:
        b = [a[n] for n in ("rows", "cols", "fmt", "codes", "scales", "x", "dt", "ld")]
        assert lib.mx_dequantize(*b, None) == status


def test_empty_launches_nothing(lib):
    for rows, cols in ((0, 32), (4, 0)):
        assert lib.mx_quantize(rows, cols, None, 2, cols, 0, 1, None, None, None) == _abi.OK
        assert lib.mx_quantize(rows, cols, None, 2, cols, 1, 1, None, None, None) == _abi.OK
        assert lib.mx_dequantize(rows, cols, 1, None, None, None, 2, cols, None) == _abi.OK
    a = _abi.RmsnormArgs(rows=0, cols=8, type=2, y=P)
    assert lib.rmsnorm_forward(ctypes.byref(a), None) == _abi.OK


def norm_args(**kw):
    a = _abi.RmsnormArgs(rows=4, cols=64, type=2, q_format=1, eps=1e-5, x=P, residual=P, weight=P, h_out=P, y=P,
                         q_codes=P, q_scales=P, rstd=P, ldx=64, ldr=64, ldh=64, ldy=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(type=4), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(y=None, q_codes=None, q_scales=None), 1), (dict(q_scales=None), 1), (dict(residual=None), 1),
    (dict(q_format=2), 1), (dict(x=None), 1), (dict(weight=None), 1), (dict(ldx=63), 1), (dict(ldy=1), 1),
    (dict(ldh=128), 1), (dict(rows=(1 << 30) + 1), 2), (dict(ldr=1 << 49), 2), (dict(x=P + 1, h_out=P + 64), 3),
    (dict(y=P + 1), 3), (dict(q_codes=P + 8), 3), (dict(rstd=P + 2), 3),
])
def test_norm_refusals(lib, kw, status):
    a = norm_args(**kw)
    assert lib.rmsnorm_forward(ctypes.byref(a), None) == status and lib.gemm_last_error()
    assert lib.rmsnorm_forward(None, None) == _abi.INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(type=0), 1), (dict(dw=None), 1), (dict(dw=P + 2), 3), (dict(dy=None), 1),
    (dict(h=None), 1), (dict(rstd=None), 1), (dict(weight=P + 1), 3), (dict(dx=None), 1), (dict(workspace=None), 1),
    (dict(workspace_bytes=4 * 64 * 4 - 1), 1), (dict(workspace=P + 4), 3), (dict(lddx=63), 1), (dict(lddres=1), 1),
    (dict(lddy=128), 1), (dict(dres=P, lddres=128), 1),
])
def test_norm_backward_refusals(lib, kw, status):
    a = _abi.RmsnormBackwardArgs(rows=4, cols=64, type=2, dy=P, h=P, weight=P, rstd=P, dres=P + 64, dx=P, dw=P,
                                 workspace=P, workspace_bytes=1 << 20, lddy=64, ldh=64, lddres=64, lddx=64)
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.rmsnorm_backward(ctypes.byref(a), None) == status and lib.gemm_last_error()


def test_backward_workspace():
    assert gep.rmsnorm_backward_workspace(0, 100) == 0
    assert gep.rmsnorm_backward_workspace(3, 100) == 3 * 100 * 4
    assert gep.rmsnorm_backward_workspace(1 << 20, 64) >= 64 * 4
    with pytest.raises(ValueError):
        gep.rmsnorm_backward_workspace(-1, 3)


def gemm_desc(**kw):
    d = _abi.MxGemmDesc(M=64, N=64, K=100, groups=0, a_format=1, b_format=0, c=2, d=2, post=2, act=4, tile=0, split=0, ldc=64,
                        ldd=64, ldp=64)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(K=0), 0), (dict(M=0), 0), (dict(c=0), 0), (dict(d=3), 0), (dict(groups=1024), 0),
    (dict(M=-1), 1), (dict(groups=-1), 1), (dict(groups=1025), 2), (dict(a_format=2), 1), (dict(b_format=-1), 1),
    (dict(d=9), 1), (dict(d=0, post=0, act=0), 1), (dict(act=5), 1), (dict(post=0), 1), (dict(tile=7), 1), (dict(tile=-1), 1), (dict(split=-1), 1), (dict(split=65), 1),
    (dict(split=2, groups=2), 2), (dict(split=2, tile=1), 2),
    (dict(N=60), 3), (dict(K=(1 << 22) + 1), 2), (dict(d=4), 2), (dict(c=5), 2), (dict(ldd=56), 1), (dict(ldd=-8), 1),
    (dict(ldp=68), 3), (dict(ldc=1 << 49), 2), (dict(M=2 ** 31 - 1, N=1 << 20, ldc=1 << 20, ldd=1 << 20, ldp=1 << 20), 2),
])
def test_gemm_create_refusals(lib, kw, status):
    h = ctypes.c_void_p()
    assert lib.mx_gemm_create(ctypes.byref(gemm_desc(**kw)), ctypes.byref(h)) == status
    if status:
        assert not h.value and lib.gemm_last_error()
    else:
        lib.mx_gemm_destroy(h)
    assert lib.mx_gemm_create(None, ctypes.byref(h)) == _abi.INVALID_ARG
    assert lib.mx_gemm_create(ctypes.byref(gemm_desc()), None) == _abi.INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(a_codes=None), 1), (dict(b_scales=None), 1), (dict(C=None), 1), (dict(D=None), 1), (dict(PostAct=None), 1),
    (dict(cu_seqlens_m=P), 1), (dict(a_codes=P + 8), 3), (dict(b_scales=P + 1), 3), (dict(D=P + 2), 3),
])
def test_gemm_run_refusals(lib, kw, status):
    h = ctypes.c_void_p()
    assert lib.mx_gemm_create(ctypes.byref(gemm_desc()), ctypes.byref(h)) == 0
    a = _abi.MxGemmArgs(P, P, P, P, P, P, P, None, None, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.mx_gemm_run(h, ctypes.byref(a), None) == status and lib.gemm_last_error()
    assert lib.mx_gemm_run(None, ctypes.byref(a), None) == _abi.INVALID_ARG
    assert lib.mx_gemm_run(h, None, None) == _abi.INVALID_ARG
    lib.mx_gemm_destroy(h)
    # a grouped plan wants its offsets; an empty problem wants nothing
    assert lib.mx_gemm_create(ctypes.byref(gemm_desc(groups=2)), ctypes.byref(h)) == 0
    a = _abi.MxGemmArgs(P, P, P, P, P, P, P, None, None, 0)
    assert lib.mx_gemm_run(h, ctypes.byref(a), None) == _abi.INVALID_ARG
    a.cu_seqlens_m = P + 2
    assert lib.mx_gemm_run(h, ctypes.byref(a), None) == _abi.ALIGNMENT
    lib.mx_gemm_destroy(h)
    assert lib.mx_gemm_create(ctypes.byref(gemm_desc(M=0)), ctypes.byref(h)) == 0
    assert lib.mx_gemm_run(h, ctypes.byref(_abi.MxGemmArgs()), None) == _abi.OK
    lib.mx_gemm_destroy(h)
    assert lib.mx_gemm_destroy(None) == _abi.OK


def test_plan_tile(lib):
    def choice(cus=256, **kw):
        h, t, n, b = ctypes.c_void_p(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
        assert lib.mx_gemm_create(ctypes.byref(gemm_desc(**kw)), ctypes.byref(h)) == 0
        assert lib.mx_gemm_plan_tile(h, cus, ctypes.byref(t), ctypes.byref(n)) == 0
        assert lib.mx_gemm_workspace(h, cus, ctypes.byref(b)) == 0
        assert lib.mx_gemm_plan_tile(h, 0, ctypes.byref(t), None) == _abi.INVALID_ARG
        assert lib.mx_gemm_workspace(h, 0, ctypes.byref(b)) == _abi.INVALID_ARG
        assert lib.mx_gemm_workspace(h, cus, None) == _abi.INVALID_ARG
        lib.mx_gemm_destroy(h)
        d = gemm_desc(**kw)
        assert b.value == (n.value * d.M * d.N * 4 if n.value > 1 else 0)
        return t.value, n.value
    wide = dict(ldc=8192, ldd=8192, ldp=8192)
    for want in range(1, 7):
        assert choice(tile=want, split=1) == (want, 1)
    assert choice(tile=2, split=3, K=4096) == (2, 3)
    assert choice(tile=3, split=7, K=4096) == (3, 4)  # 8 scale tiles, two a slice
    assert choice(tile=3, split=9, K=1000) == (3, 2)
    assert choice(tile=3, split=9, K=0) == (3, 1)
    assert choice(M=8192, N=8192, K=8192, **wide) == (_abi.MX_TILE["256"], 1)
    assert choice(M=1, N=8192, K=8192, **wide)[0] in (_abi.MX_TILE["16"], _abi.MX_TILE["16x32"])
    assert choice(M=128, N=512, K=8192, d=2, ldd=512, c=0, post=0, act=0, tile=4)[1] > 1  # few tiles, a deep product


def test_mx_tensor_refusals():
    q = gep.mx_empty(70, 100, "e4m3", device="cpu")
    c, s = q.codes, q.scales
    T = gep.MxTensor
    with pytest.raises(ValueError):
        T(c, s, "e5m2", 100)
    with pytest.raises(ValueError):
        T(c, s, "e4m3", -1)
    with pytest.raises(ValueError):
        T(c, s, "e2m1", 100)  # the row length of the other format
    with pytest.raises(ValueError):
        T(c, s, "e4m3", 129)
    with pytest.raises(TypeError):
        T(c.view(torch.int8), s, "e4m3", 100)
    with pytest.raises(ValueError):
        T(c, s[:1], "e4m3", 100)
    with pytest.raises(ValueError):
        T(c[:, ::2], s, "e4m3", 60)
    with pytest.raises(ValueError):
        T(c.t(), s, "e4m3", 100)
    with pytest.raises(ValueError):
        T(c[0], s, "e4m3", 100)
    with pytest.raises(ValueError):
        gep.mx_empty(-1, 3, "e4m3", device="cpu")
    with pytest.raises(ValueError):
        gep.mx_empty(1, 3, "fp4", device="cpu")
    with pytest.raises(ValueError):
        q.group(0)


def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 32)
    q = gep.mx_empty(4, 32, "e4m3", device="cpu")
    with pytest.raises(ValueError):
        gep.mx_quantize(x, "e4m3", out=q)
    with pytest.raises(ValueError):
        gep.mx_dequantize(q, out=x)
    with pytest.raises(ValueError):
        gep.rmsnorm(x, torch.ones(32))
    with pytest.raises(ValueError):
        gep.rmsnorm_backward(x, x, torch.ones(32), torch.ones(4))
    with pytest.raises(ValueError):
        gep.MxPlan(q, q, D=x)


def test_plan_tile_of_very_many_columns(lib):
    """A grid is launched only where its threads number below 2^32: one row and 2^27 columns go to a
    kernel of a persistent grid, and a tile asked for that cannot be launched is refused."""
    d = dict(M=1, N=1 << 27, K=32, c=0, post=0, act=0, ldd=1 << 27)
    h, t = ctypes.c_void_p(), ctypes.c_int32()
    assert lib.mx_gemm_create(ctypes.byref(gemm_desc(**d)), ctypes.byref(h)) == 0
    assert lib.mx_gemm_plan_tile(h, 256, ctypes.byref(t), None) == 0
    bn = {1: 256, 2: 128, 3: 64, 4: 32, 5: 32, 6: 16}[t.value]
    assert t.value <= 2 or (1 << 27) // bn * 512 < 1 << 32
    lib.mx_gemm_destroy(h)


@pytest.mark.parametrize("kw,status", [
    (dict(), 1), (dict(x=P + 4096, h_out=P + 8192), 1), (dict(x=P + 4096, residual=P + 8192), 1),
    (dict(cols=(1 << 24) + 1), 2),
])
def test_norm_output_overlap_refusals(lib, kw, status):
    """y in the place of x, of the residual or of h."""
    assert lib.rmsnorm_forward(ctypes.byref(norm_args(**kw)), None) == status and lib.gemm_last_error()


@pytest.mark.parametrize("packed,structure", [
    (_abi.MX_GEMM_ARGS, _abi.MxGemmArgs), (_abi.RMSNORM_ARGS, _abi.RmsnormArgs),
    (_abi.RMSNORM_BACKWARD_ARGS, _abi.RmsnormBackwardArgs)])
def test_packed_arguments(packed, structure):
    """The bytes that the binding passes are the structure's, field by field."""
    assert packed.size == ctypes.sizeof(structure)
    names = [f for f, _ in structure._fields_]
    got = structure.from_buffer_copy(packed.pack(*range(1, len(names) + 1)))
    assert [getattr(got, f) for f in names] == list(range(1, len(names) + 1))


def test_plan_choice_is_that_of_the_device_asked_for(lib):
    """The choice that a plan keeps is used for the same number of compute units only, whatever the order
    of the questions."""
    kw = dict(M=512, N=4096, K=8192, c=0, d=2, post=0, act=0, ldd=4096)
    counts = (8, 32, 256, 304, 100000)

    def ask(h, cus):
        t, n = ctypes.c_int32(), ctypes.c_int32()
        assert lib.mx_gemm_plan_tile(h, cus, ctypes.byref(t), ctypes.byref(n)) == 0
        return t.value, n.value
    fresh = []
    for cus in counts:
        h = ctypes.c_void_p()
        assert lib.mx_gemm_create(ctypes.byref(gemm_desc(**kw)), ctypes.byref(h)) == 0
        fresh.append(ask(h, cus))
        lib.mx_gemm_destroy(h)
    assert len(set(fresh)) > 1
    h = ctypes.c_void_p()
    assert lib.mx_gemm_create(ctypes.byref(gemm_desc(**kw)), ctypes.byref(h)) == 0
    for _ in range(2):
        for cus, want in zip(counts, fresh):
            assert ask(h, cus) == want and ask(h, cus) == want
    lib.mx_gemm_destroy(h)


def test_norm_without_rows(lib):
    """No rows: every matrix may be NULL, as the address of an empty one is; sizes, type, eps and format are
    looked at all the same."""
    a = _abi.RmsnormArgs(rows=0, cols=64, type=2, eps=1e-5, ldx=64, ldy=64)
    assert lib.rmsnorm_forward(ctypes.byref(a), None) == _abi.OK
    for kw in (dict(cols=0), dict(type=4), dict(eps=-1.0)):
        b = _abi.RmsnormArgs.from_buffer_copy(a)
        for k, v in kw.items():
            setattr(b, k, v)
        assert lib.rmsnorm_forward(ctypes.byref(b), None) == _abi.INVALID_ARG


class OnGpu(torch.Tensor):
    """A CPU tensor that passes the checks for one on the GPU."""
    is_cuda = True


def test_workspace_is_the_streams_own(lib, monkeypatch):
    """A plan's workspace comes from the allocator under the stream that the run goes to, whichever was
    current when the plan was made: one for each stream, and one a run in a capture."""
    import contextlib
    from gemm_epilogue_persistent_amd import mx
    current, capturing, made, used = ["first"], [False], {}, []
    pointer = {"first": 11, "second": 12, "third": 13}

    class Stream:
        def __init__(self, name):
            self.name, self.cuda_stream = name, pointer[name]

    @contextlib.contextmanager
    def under(stream):
        before, current[0] = current[0], stream.name
        yield
        current[0] = before

    def launch(device, stream, function, plan, args):
        used.append((current[0] if stream is None else stream.name, _abi.MX_GEMM_ARGS.unpack(args)[8]))

    empty = torch.empty

    def allocate(*args, **kw):
        t = empty(*args, **kw)
        made.setdefault(t.data_ptr(), []).append((current[0], t))  # (kept: no address comes twice)
        return t

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, stream: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(mx, "_current_device", lambda: None)
    monkeypatch.setattr(mx, "_raw_stream", lambda index: pointer[current[0]])
    monkeypatch.setattr(mx, "_launch", launch)
    monkeypatch.setattr(gep.MxPlan, "_cus", lambda self: 256)

    def operand(rows):
        q = gep.mx_empty(rows, 4096, "e4m3", device="cpu")
        return gep.MxTensor(q.codes.as_subclass(OnGpu), q.scales, "e4m3", 4096)

    a, b, D = operand(40), operand(64), torch.zeros(40, 64).as_subclass(OnGpu)
    plan = gep.MxPlan(a, b, None, D, tile="32", split=4)
    assert plan.workspace_bytes == 4 * 40 * 64 * 4
    monkeypatch.setattr(torch, "empty", allocate)
    plan.run(a, b, None, D, stream=Stream("second"))
    plan.run(a, b, None, D)
    current[0] = "third"
    plan.run(a, b, None, D)
    plan.run(a, b, None, D, stream=Stream("first"))
    plan.run(a, b, None, D, stream=Stream("second"))
    kept = [p for _, p in used]
    for stream, p in used:
        assert [s for s, t in made.get(p, [])] == [stream] and made[p][0][1].numel() == plan.workspace_bytes
    assert [s for s, _ in used] == ["second", "first", "third", "first", "second"]
    assert kept[3] == kept[1] and kept[4] == kept[0] and len(set(kept)) == 3
    capturing[0] = True
    plan.run(a, b, None, D)
    plan.run(a, b, None, D)
    capturing[0] = False
    plan.run(a, b, None, D)
    captured = [p for _, p in used[5:7]]
    assert len({*captured, *kept}) == 5 and used[7] == ("third", kept[2])


@pytest.mark.parametrize("rows,cols,ok", [
    (1 << 30, 1 << 24, True), ((1 << 30) + 1, 64, False), (1, (1 << 24) + 1, False), (1, 2 ** 31 - 1, False),
    (2 ** 31 - 1, 2 ** 31 - 1, False), (0, 2 ** 31 - 1, False), (5, 0, True)])
def test_backward_workspace_limits(lib, rows, cols, ok):
    """The sizes that rmsnorm_backward refuses have no workspace."""
    assert (lib.rmsnorm_backward_workspace(rows, cols) >= 0) == ok
    if not ok:
        assert lib.rmsnorm_backward_workspace(rows, cols) == -1
        with pytest.raises(ValueError):
            gep.rmsnorm_backward_workspace(rows, cols)


def test_sizes_past_32_bits(lib, monkeypatch):
    """Sizes and counts that do not fit the C ABI's 32-bit fields are refused: cut to 32 bits, 2^32 rows would be
    none, and the call would return without having written anything."""
    from gemm_epilogue_persistent_amd import mx, norm
    launch = lambda device, stream, function, *args: _abi.check(function(*args, None))  # noqa: E731
    monkeypatch.setattr(mx, "_launch", launch)
    monkeypatch.setattr(norm, "_launch", launch)
    monkeypatch.setattr(gep.MxPlan, "_cus", lambda self: 256)
    big = 1 << 32

    def matrix(*shape, dtype=torch.float16):
        return torch.empty(shape, dtype=dtype, device="meta").as_subclass(OnGpu)

    def operand(rows, k, groups=None):
        q = gep.mx_empty(rows, k, "e4m3", groups=groups, device="meta")
        return gep.MxTensor(q.codes.as_subclass(OnGpu), q.scales, "e4m3", k)

    for shape in ((big, 32), (32, big), (big + 1, 1), (1, big)):
        q = operand(*shape)
        for call in (lambda: gep.mx_quantize(matrix(*shape), "e4m3", out=q),
                     lambda: gep.mx_quantize(matrix(*shape[::-1]), "e4m3", out=q, transpose=True),
                     lambda: gep.mx_dequantize(q, out=matrix(*shape)),
                     lambda: gep.rmsnorm(matrix(*shape), matrix(shape[1]).reshape(-1), y=matrix(*shape)),
                     lambda: gep.rmsnorm_backward_workspace(*shape)):
            with pytest.raises(ValueError):
                call()
    small = operand(16, 64)
    for call in (lambda: gep.MxPlan(operand(big, 64), small, None, matrix(big, 16)),
                 lambda: gep.MxPlan(small, operand(big, 64), None, matrix(16, big)),
                 lambda: gep.MxPlan(operand(16, big), operand(16, big), None, matrix(16, 16)),
                 lambda: gep.MxPlan(small, small, None, matrix(16, 16), split=big),
                 lambda: gep.MxPlan(small, small, None, matrix(16, 16)).tile(big + 256)):
        with pytest.raises(ValueError):
            call()


def test_plain_tensors_are_no_mx_operands():
    """A tensor in the place of an MX operand is a TypeError that names it."""
    q, x = gep.mx_empty(4, 32, "e4m3", device="cpu"), torch.zeros(4, 32)
    for call in (gep.MxPlan, gep.mx_gemm):
        with pytest.raises(TypeError, match="a: an MxTensor expected"):
            call(x, q, D=x)
        with pytest.raises(TypeError, match="b: an MxTensor expected"):
            call(q, x, D=x)
    with pytest.raises(TypeError, match="b: an MxTensor expected"):
        gep.mx_gemm(q, x)
    with pytest.raises(TypeError, match="a: an MxTensor expected"):
        gep.mx_gemm(None, q)
