"""CPU tests of the FP8 and router entry points: exports, sizes, and every refusal, all of them before any HIP
call (fake pointers, no GPU)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import fp8_ref as R
import gemm_epilogue_persistent_amd as gep
from gemm_epilogue_persistent_amd import _abi

P = 4096  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        from gemm_epilogue_persistent_amd import build
        build.build()
    return _abi.load()


def test_exports_every_declared_symbol(lib):
    for header, prefix, some in ((_abi.FP8_HEADER, "fp8", {"fp8_quantize", "fp8_dequantize", "fp8_act_forward", "fp8_act_backward",
                                                           "fp8_gemm_create", "fp8_gemm_run"}),
                                 (_abi.ROUTER_HEADER, "router", {"router_balance", "router_balance_backward", "router_balance_workspace"})):
        text = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
        names = set(re.findall(r"\b(%s_[a-z0-9_]+)\s*\(" % prefix, text))
        assert some <= names
        for n in names:
            assert hasattr(lib, n), n


@pytest.mark.parametrize("rows,k", [(0, 0), (0, 5), (1, 0), (1, 1), (3, 128), (64, 512), (65, 513), (129, 1000)])
def test_storage_sizes(lib, rows, k):
    kp, nq = -(-k // 16) * 16, -(-(-(-k // 128)) // 4)
    assert lib.fp8_code_bytes(rows, k) == rows * kp
    assert lib.fp8_scale_bytes(rows, k, 0) == -(-rows // 64) * nq * 1024
    assert lib.fp8_scale_bytes(rows, k, 1) == -(-rows // 128) * nq * 16
    for tiles in (False, True):
        q = gep.fp8_empty(rows, k, tiles=tiles, device="cpu")
        assert q.codes.numel() == rows * kp and q.scales.numel() * 4 == lib.fp8_scale_bytes(rows, k, int(tiles))
        assert q.shape == (rows, k) and q.tiles == tiles and not q.scales.any()
        g = gep.fp8_empty(rows, k, tiles=tiles, groups=3, device="cpu")
        assert g.shape == (3, rows, k) and g.group(1).shape == (rows, k) and g.group(2).tiles == tiles
    assert lib.fp8_code_bytes(-1, 1) == -1 and lib.fp8_scale_bytes(1, -1, 0) == -1 and lib.fp8_scale_bytes(1, 1, 2) == -1
    assert lib.fp8_code_bytes(1 << 40, 1 << 40) == -1 and lib.fp8_scale_bytes(1 << 62, 1 << 40, 0) == -1


def test_reference():
    """The tests' own implementation against torch's e4m3 and by hand."""
    m = R.magnitudes()
    assert np.array_equal(m, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    x = np.linspace(-448, 448, 20001)
    got = R.round_code(x)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got & 127, want & 127)
    # 448 / 3 = 149.33: cut to 13 bits, 149.3125
    assert R.factor(np.array([3.0]))[0] == 149.3125 and R.factor(np.array([0.0]))[0] == 2.0 ** 126
    assert R.factor(np.array([448.0]))[0] == 1.0 and R.factor(np.array([1.75]))[0] == 256.0
    c, s = R.quantize(np.array([[3.0, -3.0, 0.0]]))
    assert c[0, :3].tolist() == [126, 254, 0] and s[0, 0] == np.float32(1 / 149.3125)
    for rows, nb, tiles in ((70, 5, False), (3, 9, True)):
        s = np.random.RandomState(1).rand(rows, nb).astype(np.float32)
        assert np.array_equal(R.load_scales(R.store_scales(s, tiles), rows, tiles)[:, :nb], s)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=-1), 1), (dict(rows=(1 << 30) + 1), 2), (dict(x=None), 1), (dict(x=P + 1), 3), (dict(dt=4), 1),
    (dict(dt=0), 1), (dict(ld=31), 1), (dict(rows=1, ld=-1), 2), (dict(ld=(1 << 48) + 1), 2), (dict(sc=2), 1), (dict(sc=-1), 1),
    (dict(codes=None), 1), (dict(codes=P + 8), 3), (dict(scales=None), 1), (dict(scales=P + 2), 3),
])
def test_quantize_refusals(lib, kw, status):
    a = dict(rows=4, cols=32, x=P, dt=_abi.DT["bf16"], ld=32, sc=0, codes=P, scales=P, codes_t=P, scales_t=P)
    a.update(kw)
    assert lib.fp8_quantize(*a.values(), None) == status and lib.gemm_last_error()
    b = [a[n] for n in ("rows", "cols", "sc", "codes", "scales", "x", "dt", "ld")]
    assert lib.fp8_dequantize(*b, None) == status
    # the same for the transposed matrix alone
    t = dict(a, codes=None, scales=None, codes_t=a["codes"], scales_t=a["scales"])
    assert lib.fp8_quantize(*t.values(), None) == status


def test_quantize_needs_an_output(lib):
    assert lib.fp8_quantize(4, 32, P, 2, 32, 0, None, None, None, None, None) == _abi.INVALID_ARG


def act_args(**kw):
    a = _abi.Fp8ActArgs(rows=4, cols=64, type=2, act=4, x=P, saved_codes=P, saved_scales=P, q_codes=P, q_scales=P, y=P + 4096, ldx=64, ldy=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=(1 << 30) + 1), 2), (dict(type=4), 1), (dict(act=5), 1), (dict(act=-1), 1), (dict(x=None), 1),
    (dict(x=P + 1), 3), (dict(ldx=63), 1), (dict(ldy=63), 1), (dict(y=P + 1), 3), (dict(saved_scales=None), 1), (dict(q_codes=None), 1),
    (dict(saved_codes=P + 4), 3), (dict(q_scales=P + 1), 3), (dict(y=P, ldy=128), 1), (dict(ldx=1 << 49), 2),
    (dict(saved_codes=None, saved_scales=None, q_codes=None, q_scales=None, y=None), 1),
])
def test_act_refusals(lib, kw, status):
    assert lib.fp8_act_forward(ctypes.byref(act_args(**kw)), None) == status and lib.gemm_last_error()
    assert lib.fp8_act_forward(None, None) == _abi.INVALID_ARG


def back_args(**kw):
    a = _abi.Fp8ActBackwardArgs(rows=4, cols=64, type=2, act=4, dy=P, saved_codes=2 * P, saved_scales=2 * P, dx=3 * P, q_codes=4 * P,
                                q_scales=4 * P, qt_codes=5 * P, qt_scales=5 * P, y=6 * P, yt_codes=7 * P, yt_scales=7 * P, lddy=64,
                                lddx=64, ldy=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


NO_GRAD = dict(dx=None, q_codes=None, q_scales=None, qt_codes=None, qt_scales=None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(rows=(1 << 30) + 1), 2), (dict(type=0), 1), (dict(act=9), 1), (dict(dy=None), 1), (dict(saved_codes=None), 1),
    (dict(saved_scales=2 * P + 1), 3), (dict(saved_codes=2 * P + 8), 3), (dict(q_scales=None), 1), (dict(qt_codes=None), 1),
    (dict(yt_scales=None), 1), (dict(qt_codes=5 * P + 1), 3), (dict(lddy=63), 1), (dict(lddx=1), 1), (dict(ldy=-1), 2), (dict(dx=P, lddx=72), 1),
    (dict(y=P), 1), (dict(y=3 * P), 1), (dict(q_codes=2 * P), 1), (dict(yt_codes=5 * P), 1), (dict(dx=2 * P), 1), (NO_GRAD, 1),
    (dict(NO_GRAD, dy=None, y=None, yt_codes=None, yt_scales=None), 1), (dict(dy=P + 1), 3),
])
def test_act_backward_refusals(lib, kw, status):
    assert lib.fp8_act_backward(ctypes.byref(back_args(**kw)), None) == status and lib.gemm_last_error()
    assert lib.fp8_act_backward(None, None) == _abi.INVALID_ARG


def test_empty_launches_nothing(lib):
    for rows, cols in ((0, 32), (4, 0)):
        for sc in (0, 1):
            assert lib.fp8_quantize(rows, cols, None, 2, cols, sc, None, None, None, None, None) == _abi.OK
            assert lib.fp8_dequantize(rows, cols, sc, None, None, None, 2, cols, None) == _abi.OK
        assert lib.fp8_act_forward(ctypes.byref(_abi.Fp8ActArgs(rows=rows, cols=cols, type=2)), None) == _abi.OK
        assert lib.fp8_act_backward(ctypes.byref(_abi.Fp8ActBackwardArgs(rows=rows, cols=cols, type=2)), None) == _abi.OK
    a = _abi.RouterBalanceBackwardArgs(batch=0, tokens=4, experts=8, k=2, type=2)
    assert lib.router_balance_backward(ctypes.byref(a), None) == _abi.OK


def gemm_desc(**kw):
    d = _abi.Fp8GemmDesc(M=64, N=64, K=100, groups=0, b_scaling=1, c=2, d=2, post=2, act=4, tile=0, split=0, ldc=64, ldd=64, ldp=64)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(K=0), 0), (dict(M=0), 0), (dict(c=0), 0), (dict(d=3), 0), (dict(groups=1024), 0), (dict(b_scaling=0), 0),
    (dict(M=-1), 1), (dict(groups=-1), 1), (dict(groups=1025), 2), (dict(b_scaling=2), 1), (dict(b_scaling=-1), 1),
    (dict(d=9), 1), (dict(d=0, post=0, act=0), 1), (dict(act=5), 1), (dict(post=0), 1), (dict(tile=7), 1), (dict(tile=-1), 1),
    (dict(split=-1), 1), (dict(split=65), 1), (dict(split=2, groups=2), 2), (dict(split=2, tile=1), 2),
    (dict(N=60), 3), (dict(K=(1 << 22) + 1), 2), (dict(d=4), 2), (dict(c=5), 2), (dict(ldd=56), 1), (dict(ldd=-8), 1),
    (dict(ldp=68), 3), (dict(ldc=1 << 49), 2), (dict(M=2 ** 31 - 1, N=1 << 20, ldc=1 << 20, ldd=1 << 20, ldp=1 << 20), 2),
])
def test_gemm_create_refusals(lib, kw, status):
    h = ctypes.c_void_p()
    assert lib.fp8_gemm_create(ctypes.byref(gemm_desc(**kw)), ctypes.byref(h)) == status
    if status:
        assert not h.value and b"fp8_gemm_create" in lib.gemm_last_error()
    else:
        lib.fp8_gemm_destroy(h)
    assert lib.fp8_gemm_create(None, ctypes.byref(h)) == _abi.INVALID_ARG
    assert lib.fp8_gemm_create(ctypes.byref(gemm_desc()), None) == _abi.INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(a_codes=None), 1), (dict(b_scales=None), 1), (dict(C=None), 1), (dict(D=None), 1), (dict(PostAct=None), 1),
    (dict(cu_seqlens_m=P), 1), (dict(a_codes=P + 8), 3), (dict(b_scales=P + 1), 3), (dict(D=P + 2), 3),
    (dict(D=2 * P, PostAct=2 * P), 1),
])
def test_gemm_run_refusals(lib, kw, status):
    h = ctypes.c_void_p()
    assert lib.fp8_gemm_create(ctypes.byref(gemm_desc()), ctypes.byref(h)) == 0
    a = _abi.Fp8GemmArgs(P, P, P, P, P, P, 2 * P, None, None, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.fp8_gemm_run(h, ctypes.byref(a), None) == status and b"fp8_gemm_run" in lib.gemm_last_error()
    assert lib.fp8_gemm_run(None, ctypes.byref(a), None) == _abi.INVALID_ARG
    assert lib.fp8_gemm_run(h, None, None) == _abi.INVALID_ARG
    lib.fp8_gemm_destroy(h)
    assert lib.fp8_gemm_create(ctypes.byref(gemm_desc(groups=2)), ctypes.byref(h)) == 0
    a = _abi.Fp8GemmArgs(P, P, P, P, P, P, 2 * P, None, None, 0)
    assert lib.fp8_gemm_run(h, ctypes.byref(a), None) == _abi.INVALID_ARG
    a.cu_seqlens_m = P + 2
    assert lib.fp8_gemm_run(h, ctypes.byref(a), None) == _abi.ALIGNMENT
    lib.fp8_gemm_destroy(h)
    assert lib.fp8_gemm_create(ctypes.byref(gemm_desc(M=0)), ctypes.byref(h)) == 0
    assert lib.fp8_gemm_run(h, ctypes.byref(_abi.Fp8GemmArgs()), None) == _abi.OK
    lib.fp8_gemm_destroy(h)
    assert lib.fp8_gemm_destroy(None) == _abi.OK


def test_plan_tile(lib):
    def choice(cus=256, **kw):
        h, t, n, b = ctypes.c_void_p(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
        assert lib.fp8_gemm_create(ctypes.byref(gemm_desc(**kw)), ctypes.byref(h)) == 0
        assert lib.fp8_gemm_plan_tile(h, cus, ctypes.byref(t), ctypes.byref(n)) == 0
        assert lib.fp8_gemm_workspace(h, cus, ctypes.byref(b)) == 0
        assert lib.fp8_gemm_plan_tile(h, 0, ctypes.byref(t), None) == _abi.INVALID_ARG
        assert lib.fp8_gemm_workspace(h, 0, ctypes.byref(b)) == _abi.INVALID_ARG
        assert lib.fp8_gemm_workspace(h, cus, None) == _abi.INVALID_ARG
        lib.fp8_gemm_destroy(h)
        d = gemm_desc(**kw)
        assert b.value == (n.value * d.M * d.N * 4 if n.value > 1 else 0)
        return t.value, n.value
    for want in range(1, 7):
        assert choice(tile=want, split=1) == (want, 1)
    assert choice(tile=2, split=3, K=4096) == (2, 3)
    assert choice(tile=3, split=9, K=1000) == (3, 2)
    wide = dict(ldc=8192, ldd=8192, ldp=8192)
    assert choice(M=8192, N=8192, K=8192, **wide) == (_abi.FP8_TILE["256"], 1)
    assert choice(M=1, N=8192, K=8192, **wide) == (_abi.FP8_TILE["16"], 1)
    assert choice(M=256, N=4096, K=4096, **wide) == (_abi.FP8_TILE["64"], 1)
    assert choice(M=512, N=512, K=8192, **wide)[1] > 1 and choice(M=512, N=512, K=8192, groups=4, **wide)[1] == 1


def balance_args(**kw):
    a = _abi.RouterBalanceArgs(batch=2, tokens=5, experts=8, k=2, type=3, scores=0, index_bytes=8, coef=1.0, logits=P, chosen=P, mask=P,
                               counts=P, valid=P, cu_seqlens=P, probs=P, loss=P, workspace=P, workspace_bytes=1 << 20, logits_ld=8,
                               logits_batch=40)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(tokens=-1), 1), (dict(experts=0), 1), (dict(experts=2049), 2), (dict(k=0), 1), (dict(k=9), 1),
    (dict(batch=65536), 2), (dict(batch=60000, tokens=60000), 2), (dict(type=4), 1), (dict(scores=2), 1), (dict(index_bytes=2), 1),
    (dict(logits=None), 1), (dict(logits=P + 1), 3), (dict(logits_ld=7), 1), (dict(logits_batch=39), 1), (dict(logits_ld=-1), 2),
    (dict(logits_batch=1 << 49), 2), (dict(chosen=None), 1), (dict(chosen=P + 4), 3), (dict(counts=None), 1), (dict(valid=None), 1),
    (dict(probs=None), 1), (dict(loss=None), 1), (dict(cu_seqlens=P + 2), 3), (dict(loss=P + 1), 3), (dict(workspace=None), 1),
    (dict(workspace_bytes=16), 1), (dict(workspace=P + 8), 3),
])
def test_balance_refusals(lib, kw, status):
    assert lib.router_balance(ctypes.byref(balance_args(**kw)), None) == status and lib.gemm_last_error()
    assert lib.router_balance(None, None) == _abi.INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(experts=2049), 2), (dict(k=9), 1), (dict(type=0), 1), (dict(scores=-1), 1), (dict(logits=None), 1),
    (dict(dlogits=None), 1), (dict(dlogits=P + 2), 3), (dict(dlogits_ld=7), 1), (dict(dlogits_batch=1), 1), (dict(counts=None), 1),
    (dict(valid=None), 1), (dict(grad=P + 1), 3), (dict(dlogits=P, dlogits_ld=9, dlogits_batch=80), 1), (dict(dlogits=P, dlogits_batch=80), 1),
])
def test_balance_backward_refusals(lib, kw, status):
    a = _abi.RouterBalanceBackwardArgs(batch=2, tokens=5, experts=8, k=2, type=3, scores=0, coef=1.0, logits=P, mask=None, counts=P, valid=P,
                                       grad=P, dlogits=2 * P, logits_ld=8, logits_batch=40, dlogits_ld=8, dlogits_batch=40)
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.router_balance_backward(ctypes.byref(a), None) == status and lib.gemm_last_error()
    assert lib.router_balance_backward(None, None) == _abi.INVALID_ARG


def test_balance_workspace(lib):
    for b, t, e in ((0, 5, 8), (1, 0, 8), (1, 16, 8), (8, 4096, 256), (65535, 1, 1), (1, 2 ** 31 - 1, 1), (65535, 32767, 2048)):
        n = gep.router_balance_workspace(b, t, e)
        # (the largest: 65535 sequences x 2048 experts x 8 bytes, 2^30 - 2^14, and 4 bytes for each 64 experts)
        assert 0 < n < 1 << 31
    assert gep.router_balance_workspace(1, 16, 8) < 4096
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, 0), (1, 1, 2049), (65536, 1, 1)):
        with pytest.raises(ValueError):
            gep.router_balance_workspace(*bad)
    with pytest.raises(ValueError):
        gep.router_balance_workspace(1, 1 << 32, 8)


@pytest.mark.parametrize("packed,structure", [
    (_abi.MX_GEMM_ARGS, _abi.Fp8GemmArgs), (_abi.FP8_ACT_ARGS, _abi.Fp8ActArgs), (_abi.FP8_ACT_BACKWARD_ARGS, _abi.Fp8ActBackwardArgs),
    (_abi.ROUTER_BALANCE_ARGS, _abi.RouterBalanceArgs), (_abi.ROUTER_BALANCE_BACKWARD_ARGS, _abi.RouterBalanceBackwardArgs)])
def test_packed_arguments(packed, structure):
    """The bytes that the binding passes are the structure's, field by field."""
    assert packed.size == ctypes.sizeof(structure)
    names = [f for f, _ in structure._fields_]
    got = structure.from_buffer_copy(packed.pack(*range(1, len(names) + 1)))
    assert [getattr(got, f) for f in names] == list(range(1, len(names) + 1))


def test_fp8_tensor_refusals():
    q, w = gep.fp8_empty(70, 100, device="cpu"), gep.fp8_empty(70, 100, tiles=True, device="cpu")
    c, s = q.codes, q.scales
    T = gep.Fp8Tensor
    assert not T(c, s, 100).tiles and T(c, w.scales, 100).tiles and T(c, s, 112).k == 112
    for args in ((c, s, -1), (c, s, 113), (c, s, 96), (c, s[:1], 100), (c, w.scales[:, :1], 100), (c[:, ::2], s, 50), (c.t(), s, 100), (c[0], s, 100)):
        with pytest.raises(ValueError):
            T(*args)
    with pytest.raises(TypeError):
        T(c.view(torch.int8), s, 100)
    with pytest.raises(TypeError):
        T(c, s.double(), 100)
    with pytest.raises(ValueError):
        gep.fp8_empty(-1, 3, device="cpu")
    with pytest.raises(ValueError):
        q.group(0)


def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 32)
    q = gep.fp8_empty(4, 32, device="cpu")
    for call in (lambda: gep.fp8_quantize(x, out=q), lambda: gep.fp8_quantize(x), lambda: gep.fp8_dequantize(q, out=x),
                 lambda: gep.Fp8Plan(q, q, D=x), lambda: gep.fp8_act(x, "silu", saved=q), lambda: gep.fp8_act_backward(x, q, "silu", dx=x),
                 lambda: gep.router_balance(x, torch.zeros(4, 2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()


class OnGpu(torch.Tensor):
    """A CPU tensor that passes the checks for one on the GPU."""
    is_cuda = True


def test_sizes_past_32_bits(lib, monkeypatch):
    """Sizes that 32 bits do not hold are refused by name, and never cut."""
    from gemm_epilogue_persistent_amd import fp8, mx, router

    def never(*a):
        raise AssertionError("launched")
    for m in (fp8, mx, router):
        monkeypatch.setattr(m, "_launch", never)
    many = 1 << 32
    x = torch.empty(0).as_subclass(OnGpu)
    wide = torch.empty((0, many)).as_subclass(OnGpu)
    with pytest.raises(ValueError, match="2\\^31"):
        gep.fp8_quantize(wide, out=gep.Fp8Tensor(torch.empty((0, many), dtype=torch.uint8).as_subclass(OnGpu),
                                                 torch.empty((0, many // 512, 64, 4)).as_subclass(OnGpu), many))
    q = gep.Fp8Tensor(torch.empty((0, many), dtype=torch.uint8).as_subclass(OnGpu), torch.empty((0, many // 512, 64, 4)).as_subclass(OnGpu), many)
    with pytest.raises(ValueError):
        gep.fp8_dequantize(q, out=wide)
    with pytest.raises(ValueError):
        gep.fp8_act(wide, "silu", y=wide)
    with pytest.raises(ValueError):
        gep.fp8_act_backward(None, q, "silu", y=wide)
    with pytest.raises(ValueError):
        gep.router_balance(torch.empty((0, many, 8)).as_subclass(OnGpu), torch.empty((0, many, 2), dtype=torch.int64))
    del x


def test_one_matrix_twice(lib):
    """Two outputs at one address are refused."""
    assert lib.fp8_quantize(128, 128, P, 2, 128, 0, 2 * P, 2 * P, 2 * P, 2 * P, None) == _abi.INVALID_ARG
    assert lib.fp8_act_forward(ctypes.byref(act_args(q_codes=2 * P, saved_codes=2 * P)), None) == _abi.INVALID_ARG
    with pytest.raises(TypeError):
        gep.fp8_dequantize(None)


def test_sequence_strides(lib):
    """Sequences that overlap are refused, whatever their strides' product; those that alternate row by row are not (the
    refusal here is that of the workspace, which comes later)."""
    big = 1 << 48
    for kw in (dict(logits_ld=big, logits_batch=big), dict(logits_ld=15, logits_batch=8), dict(logits_ld=16, logits_batch=7),
               dict(tokens=2 ** 30 - 1, batch=2, k=1, logits_ld=big, logits_batch=big)):
        assert lib.router_balance(ctypes.byref(balance_args(**kw)), None) == _abi.INVALID_ARG
        assert b"sequences of logits overlap" in lib.gemm_last_error() or b"rows of logits" in lib.gemm_last_error()
    for kw in (dict(logits_ld=16, logits_batch=8), dict(logits_ld=8, logits_batch=40)):
        assert lib.router_balance(ctypes.byref(balance_args(workspace=None, **kw)), None) == _abi.INVALID_ARG
        assert b"workspace" in lib.gemm_last_error()


def test_workspace_of_many_tokens():
    """Sharing out 2^31 - 1 tokens is 64-bit arithmetic: 256 workgroups' sums, not one for each 256 tokens."""
    assert gep.router_balance_workspace(1, 2 ** 31 - 1, 8) < 1 << 20
