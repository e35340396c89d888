"""ctypes view of include/gemm_mi355x.h (argument marshalling only)."""
import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgemm_mi355x.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "gemm_mi355x.h")

OK, INVALID_ARG, UNSUPPORTED, ALIGNMENT, HIP_ERROR, NO_MEMORY = range(6)
DT = {"none": 0, "f16": 1, "bf16": 2, "f32": 3, "e4m3": 4, "e5m2": 5}
ROW, COL = 0, 1
ACT = {"none": 0, "relu": 1, "relu_sq": 2, "gelu_tanh": 3, "silu": 4}
MX_FORMAT = {"e2m1": 0, "e4m3": 1}
MX_TILE = {"auto": 0, "256": 1, "128": 2, "32x64": 3, "32": 4, "16x32": 5, "16": 6}
MX_HEADER = os.path.join(os.path.dirname(HERE), "include", "mx_mi355x.h")


class GemmDesc(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("L", ctypes.c_int32),
        ("a", ctypes.c_int32), ("b", ctypes.c_int32), ("c", ctypes.c_int32), ("d", ctypes.c_int32),
        ("post", ctypes.c_int32),
        ("a_major", ctypes.c_int32), ("b_major", ctypes.c_int32), ("c_major", ctypes.c_int32),
        ("d_major", ctypes.c_int32), ("post_major", ctypes.c_int32),
        ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldc", ctypes.c_int64),
        ("ldd", ctypes.c_int64), ("ldp", ctypes.c_int64),
        ("sa", ctypes.c_int64), ("sb", ctypes.c_int64), ("sc", ctypes.c_int64),
        ("sd", ctypes.c_int64), ("sp", ctypes.c_int64),
        ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
        ("act", ctypes.c_int32), ("varlen_m", ctypes.c_int32),
        ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
        ("group_m", ctypes.c_int32), ("max_ctas", ctypes.c_int32), ("xcd_remap", ctypes.c_int32),
        ("tail_split", ctypes.c_int32), ("raster_order", ctypes.c_int32), ("dact", ctypes.c_int32),
        ("varlen_k", ctypes.c_int32), ("gather_a", ctypes.c_int32), ("gather_rows", ctypes.c_int64),
    ]


class GemmArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("A", "B", "C", "D", "PostAct", "alpha_dev", "beta_dev",
                                               "cu_seqlens_m", "cu_seqlens_k", "a_idx", "tile_counters")]


class MxGemmDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "groups", "a_format", "b_format", "c", "d", "post",
                                              "act", "tile", "split")] + [
        (n, ctypes.c_int64) for n in ("ldc", "ldd", "ldp")]


class MxGemmArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("a_codes", "a_scales", "b_codes", "b_scales", "C", "D", "PostAct",
                                               "cu_seqlens_m", "workspace")] + [
        ("workspace_bytes", ctypes.c_int64)]


class RmsnormArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "cols", "type", "q_format")] + [("eps", ctypes.c_float)] + [
        (n, ctypes.c_void_p) for n in ("x", "residual", "weight", "h_out", "y", "q_codes", "q_scales", "rstd")] + [
        (n, ctypes.c_int64) for n in ("ldx", "ldr", "ldh", "ldy")]


class RmsnormBackwardArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "cols", "type")] + [
        (n, ctypes.c_void_p) for n in ("dy", "h", "weight", "rstd", "dres", "dx", "dw", "workspace")] + [
        (n, ctypes.c_int64) for n in ("workspace_bytes", "lddy", "ldh", "lddres", "lddx")]


# The same structures as bytes, filled in a quarter of a ctypes structure's time (0.4 instead of 1.3
# us, of 5 to 10 that a call takes); NULL is 0.
MX_GEMM_ARGS = struct.Struct("@9Pq")
RMSNORM_ARGS = struct.Struct("@4if8P4q")
RMSNORM_BACKWARD_ARGS = struct.Struct("@3i8P5q")


def int32(name, value):
    """value as an int32 field takes it (ctypes would cut it to 32 bits without a word)."""
    value = int(value)
    if not -(1 << 31) <= value < 1 << 31:
        raise ValueError(f"{name} = {value} does not fit 32 bits")
    return value


class GemmError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{message} (status {status})")
        self.status = status


_lib = None


def load():
    """Load the HIP library; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with gemm_epilogue_persistent_amd/build.py")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, u32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32
        lib.gemm_create.restype = ctypes.c_int
        lib.gemm_create.argtypes = [ctypes.POINTER(GemmDesc), ctypes.POINTER(vp)]
        lib.gemm_run.restype = ctypes.c_int
        lib.gemm_run.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.gemm_run_logged.restype = ctypes.c_int
        lib.gemm_run_logged.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp]
        lib.gemm_run_dynamic.restype = ctypes.c_int
        lib.gemm_run_dynamic.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp]
        lib.gemm_run_dynamic_noalloc.restype = ctypes.c_int
        lib.gemm_run_dynamic_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.gemm_check_cu_seqlens.restype = ctypes.c_int
        lib.gemm_check_cu_seqlens.argtypes = [vp, i32, i32, i32, vp, vp]
        lib.gemm_run_ex.restype = ctypes.c_int
        lib.gemm_run_ex.argtypes = [vp, ctypes.POINTER(GemmArgs), vp]
        lib.gemm_destroy.restype = ctypes.c_int
        lib.gemm_destroy.argtypes = [vp]
        lib.gemm_plan_grid.restype = ctypes.c_int
        lib.gemm_plan_grid.argtypes = [vp, i32, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                       ctypes.POINTER(i32), ctypes.POINTER(i32),
                                       ctypes.POINTER(i64), ctypes.POINTER(i32)]
        lib.gemm_plan_raster.restype = ctypes.c_int
        lib.gemm_plan_raster.argtypes = [vp, ctypes.POINTER(i32)]
        lib.gemm_fastdivmod_params.restype = ctypes.c_int
        lib.gemm_fastdivmod_params.argtypes = [u32, ctypes.POINTER(u32), ctypes.POINTER(u32)]
        lib.gemm_fastdivmod_check.restype = ctypes.c_int
        lib.gemm_fastdivmod_check.argtypes = [u32, u32, u32, vp, vp]
        lib.mx_code_bytes.restype = i64
        lib.mx_code_bytes.argtypes = [i64, i64, i32]
        lib.mx_scale_bytes.restype = i64
        lib.mx_scale_bytes.argtypes = [i64, i64]
        lib.mx_quantize.restype = ctypes.c_int
        lib.mx_quantize.argtypes = [i32, i32, vp, i32, i64, i32, i32, vp, vp, vp]
        lib.mx_dequantize.restype = ctypes.c_int
        lib.mx_dequantize.argtypes = [i32, i32, i32, vp, vp, vp, i32, i64, vp]
        lib.rmsnorm_forward.restype = ctypes.c_int
        lib.rmsnorm_forward.argtypes = [vp, vp]
        lib.rmsnorm_backward.restype = ctypes.c_int
        lib.rmsnorm_backward.argtypes = [vp, vp]
        lib.rmsnorm_backward_workspace.restype = i64
        lib.rmsnorm_backward_workspace.argtypes = [i32, i32]
        lib.mx_gemm_create.restype = ctypes.c_int
        lib.mx_gemm_create.argtypes = [ctypes.POINTER(MxGemmDesc), ctypes.POINTER(vp)]
        lib.mx_gemm_run.restype = ctypes.c_int
        lib.mx_gemm_run.argtypes = [vp, vp, vp]
        lib.mx_gemm_destroy.restype = ctypes.c_int
        lib.mx_gemm_destroy.argtypes = [vp]
        lib.mx_gemm_plan_tile.restype = ctypes.c_int
        lib.mx_gemm_plan_tile.argtypes = [vp, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]
        lib.mx_gemm_workspace.restype = ctypes.c_int
        lib.mx_gemm_workspace.argtypes = [vp, i32, ctypes.POINTER(i64)]
        lib.gemm_status_string.restype = ctypes.c_char_p
        lib.gemm_status_string.argtypes = [ctypes.c_int]
        lib.gemm_last_error.restype = ctypes.c_char_p
        lib.gemm_last_error.argtypes = []
        _lib = lib
    return _lib


def check(status):
    if status != OK:
        lib = load()
        msg = lib.gemm_last_error().decode() or lib.gemm_status_string(status).decode()
        raise GemmError(status, msg)
