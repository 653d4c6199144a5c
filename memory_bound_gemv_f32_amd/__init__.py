"""Python binding of libgemv (dense GEMV for MI355X / gfx950).

Marshalling only: every step of the computation runs in the HIP kernels of
``libgemv.so``; this module passes device pointers, sizes and the current
HIP stream through ctypes.  There is no CPU fallback: importing this package
without a built ``libgemv.so`` raises ``ImportError``.

Two levels:

* the C ABI under the same names (``gemv_f32``, ``gemv_f16``, ``gemv_bf16``,
  ``gemv_batched_*``, ``gemv_multi_*``, ``gemv_gate_up_silu_*``,
  ``gemv_splitk_*``, ``gemv_q8_*``, ``gemv_fp8_*``, ``gemv_kv_*``, ``gemv_plan``,
  ``gemv_run_family``, ...), taking integer addresses and returning the
  ``gemv_status_t`` code;
* tensor helpers ``gemv``, ``gemv_batched``, ``gemv_multi``,
  ``gemv_gate_up_silu``, ``gemv_splitk`` and ``gemv_q8`` that check dtype, shape,
  strides and device, call the matching entry point on
  ``torch.cuda.current_stream()`` and raise ``GemvError`` on a failure code;
  ``gemv_fp8_quantise`` and ``gemv_fp8`` (e4m3 with a scale per block of 128)
  and ``gemv_kv_append`` and ``gemv_kv_attend`` (a paged 8-bit key/value cache,
  ``KVCache``) do so on the current stream of their tensors' device.

Layout of the tensor helpers: ``A`` is (M, K) with unit column stride and row
stride ``lda = A.stride(0) >= K`` (so a column slice of a wider matrix works);
``x`` is (K,); for the batched form ``X`` is (nvec, K) contiguous, which is the
K×nvec column-major matrix of the C ABI, and the result is (nvec, M)
contiguous, i.e. Y as M×nvec column-major.
"""

from __future__ import annotations

import ctypes
import functools
import os
from pathlib import Path

# torch ships its own HIP runtime under the same soname (libamdhip64.so.7) as
# the system one that libgemv is linked against.  Whichever loads first is the
# one the process uses, so torch goes first: libgemv then launches on the
# runtime that owns torch's streams and allocations.
try:
    import torch as _torch_runtime  # noqa: F401
except ImportError:  # a C-only user of the library has no torch
    _torch_runtime = None

PACKAGE = Path(__file__).resolve().parent
# LIBGEMV_LIBRARY: another build of the same library (e.g. for comparing two
# builds in one process tree); the in-tree build by default
LIBRARY = Path(os.environ.get("LIBGEMV_LIBRARY", PACKAGE / "libgemv.so"))

if not LIBRARY.exists():
    raise ImportError(
        f"{LIBRARY} is not built; run `python memory_bound_gemv_f32_amd/build.py` "
        "(there is no fallback implementation)")

_lib = ctypes.CDLL(str(LIBRARY))

GEMV_SUCCESS = 0
GEMV_ERROR_INVALID_VALUE = 1
GEMV_ERROR_LAUNCH_FAILURE = 2

DTYPE_F32, DTYPE_F16, DTYPE_BF16 = 0, 1, 2
DTYPE_CODES = {"f32": DTYPE_F32, "f16": DTYPE_F16, "bf16": DTYPE_BF16}

FAMILY_AUTO = -1
FAMILY_ROWS_PER_WAVE = 0
FAMILY_WAVE_PER_ROW = 1
FAMILY_GROUP_PER_ROW = 2
FAMILY_BATCHED = 3
FAMILY_BATCHED_MFMA = 4
FAMILY_GATED_SILU = 5
FAMILY_SPLIT_K = 6
MAX_SEGMENTS = 8
FAMILY_NAMES = {
    FAMILY_ROWS_PER_WAVE: "rows_per_wave",
    FAMILY_WAVE_PER_ROW: "wave_per_row",
    FAMILY_GROUP_PER_ROW: "group_per_row",
    FAMILY_BATCHED: "batched",
    FAMILY_BATCHED_MFMA: "batched_mfma",
    FAMILY_GATED_SILU: "gated_silu",
    FAMILY_SPLIT_K: "split_k",
}


class GemvPlan(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int) for name in (
        "family", "vector_loads", "chunk_elems", "lanes_per_row",
        "rows_per_wave", "row_tiles", "waves_per_group", "rows_per_group",
        "batch", "passes", "block", "lds_bytes", "splits", "slice_elems",
        "x_in_registers", "rounding_chain", "column_blocks")] + [
        ("grid", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class GemvSegment(ctypes.Structure):
    """gemv_segment_t: one matrix of a multi-GEMV."""
    _fields_ = [("A", ctypes.c_void_p), ("lda", ctypes.c_int), ("M", ctypes.c_int),
                ("bias", ctypes.c_void_p), ("y", ctypes.c_void_p)]


_vp, _i, _st = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p


def _bind(name, argtypes, restype=ctypes.c_int):
    fn = getattr(_lib, name)
    fn.argtypes = argtypes
    fn.restype = restype
    return fn


gemv_status_string = _bind("gemv_status_string", [_i], ctypes.c_char_p)
gemv_last_hip_error = _bind("gemv_last_hip_error", [])
gemv_last_hip_error_string = _bind("gemv_last_hip_error_string", [], ctypes.c_char_p)
gemv_f32 = _bind("gemv_f32", [_vp, _i, _vp, _vp, _vp, _i, _i, _st])
gemv_f16 = _bind("gemv_f16", [_vp, _i, _vp, _vp, _vp, _i, _i, _st])
gemv_bf16 = _bind("gemv_bf16", [_vp, _i, _vp, _vp, _vp, _i, _i, _st])
gemv_batched_f16 = _bind("gemv_batched_f16", [_vp, _i, _vp, _vp, _vp, _i, _i, _i, _st])
gemv_batched_bf16 = _bind("gemv_batched_bf16", [_vp, _i, _vp, _vp, _vp, _i, _i, _i, _st])
gemv_multi_f32 = _bind("gemv_multi_f32", [ctypes.POINTER(GemvSegment), _i, _vp, _i, _st])
gemv_multi_f16 = _bind("gemv_multi_f16", [ctypes.POINTER(GemvSegment), _i, _vp, _i, _st])
gemv_multi_bf16 = _bind("gemv_multi_bf16", [ctypes.POINTER(GemvSegment), _i, _vp, _i, _st])
gemv_gate_up_silu_f32 = _bind("gemv_gate_up_silu_f32", [_vp, _vp, _i, _vp, _vp, _i, _i, _st])
gemv_gate_up_silu_f16 = _bind("gemv_gate_up_silu_f16", [_vp, _vp, _i, _vp, _vp, _i, _i, _st])
gemv_gate_up_silu_bf16 = _bind("gemv_gate_up_silu_bf16", [_vp, _vp, _i, _vp, _vp, _i, _i, _st])
_sz = ctypes.c_size_t
gemv_splitk_workspace_size = _bind("gemv_splitk_workspace_size", [_i, _i, _i, _i, ctypes.POINTER(_sz)])
gemv_splitk_f32 = _bind("gemv_splitk_f32", [_vp, _i, _vp, _vp, _vp, _i, _i, _i, _vp, _sz, _st])
gemv_splitk_f16 = _bind("gemv_splitk_f16", [_vp, _i, _vp, _vp, _vp, _i, _i, _i, _vp, _sz, _st])
gemv_splitk_bf16 = _bind("gemv_splitk_bf16", [_vp, _i, _vp, _vp, _vp, _i, _i, _i, _vp, _sz, _st])
gemv_splitk_noalloc = _bind("gemv_splitk_noalloc", [_i, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _st])
NOALLOC_SCRATCH_BYTES = 256 * 1024
gemv_q8_f32 = _bind("gemv_q8_f32", [_vp, _i, _vp, _vp, _vp, _vp, _i, _i, _st])
gemv_q8_f16 = _bind("gemv_q8_f16", [_vp, _i, _vp, _vp, _vp, _vp, _i, _i, _st])
gemv_q8_bf16 = _bind("gemv_q8_bf16", [_vp, _i, _vp, _vp, _vp, _vp, _i, _i, _st])
gemv_q8_run_family = _bind("gemv_q8_run_family", [_i, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _st])
gemv_plan_q8 = _bind("gemv_plan_q8", [_i, _i, _i, _i, _vp, _vp, _i, ctypes.POINTER(GemvPlan)])
gemv_read_probe = _bind("gemv_read_probe", [_vp, _sz, _vp, _st])
gemv_read_probe_variant = _bind("gemv_read_probe_variant",
                                [_vp, _sz, _vp, _i, _i, _i, _i, _vp, _sz, _st])
gemv_plan = _bind("gemv_plan", [_i, _i, _i, _i, _i, _vp, _vp, _i, ctypes.POINTER(GemvPlan)])
gemv_plan_splitk = _bind("gemv_plan_splitk", [_i, _i, _i, _i, _i, _vp, _vp, ctypes.POINTER(GemvPlan)])
gemv_run_family = _bind("gemv_run_family", [_i, _i, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _st])
gemv_test_refused_launch = _bind("gemv_test_refused_launch", [_st])

FP8_BLOCK = 128
_MOST = 0x7fffffff  # what an int argument holds
KV_BLOCK = 16
KV_INT8, KV_E4M3 = 0, 1


class KvCacheStruct(ctypes.Structure):
    """gemv_kv_cache_t."""
    _fields_ = [(name, ctypes.c_int) for name in ("format", "pages", "heads", "page_size", "dim")] + [
        (name, ctypes.c_void_p) for name in ("k", "v", "k_scale", "v_scale")]


class KvBatchStruct(ctypes.Structure):
    """gemv_kv_batch_t."""
    _fields_ = [("sequences", ctypes.c_int), ("table", ctypes.c_void_p),
                ("table_pitch", ctypes.c_int), ("table_width", ctypes.c_int),
                ("seq_lens", ctypes.c_void_p), ("starts", ctypes.c_void_p)]


_cache_p, _batch_p = ctypes.POINTER(KvCacheStruct), ctypes.POINTER(KvBatchStruct)
_quantise_args = [_vp, _i, _vp, _i, _vp, _i, _i, _i, _i, _st]
gemv_fp8_quantise_f32 = _bind("gemv_fp8_quantise_f32", _quantise_args)
gemv_fp8_quantise_f16 = _bind("gemv_fp8_quantise_f16", _quantise_args)
gemv_fp8_quantise_bf16 = _bind("gemv_fp8_quantise_bf16", _quantise_args)
_fp8_args = [_vp, _i, _vp, _i, _vp, _i, _vp, _i, _vp, _vp, _i, _i, _i, _i, _st]
gemv_fp8_f32 = _bind("gemv_fp8_f32", _fp8_args)
gemv_fp8_f16 = _bind("gemv_fp8_f16", _fp8_args)
gemv_fp8_bf16 = _bind("gemv_fp8_bf16", _fp8_args)
_append_args = [_cache_p, _vp, _i, _vp, _i, _i, _batch_p, _st]
gemv_kv_append_f32 = _bind("gemv_kv_append_f32", _append_args)
gemv_kv_append_f16 = _bind("gemv_kv_append_f16", _append_args)
gemv_kv_append_bf16 = _bind("gemv_kv_append_bf16", _append_args)
gemv_kv_attend_workspace_size = _bind("gemv_kv_attend_workspace_size",
                                      [_i, _i, _i, _i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_sz)])
_attend_args = [_cache_p, _vp, _i, _vp, _i, _i, _i, _batch_p, ctypes.c_float, _i, _i, _vp, _sz, _st]
gemv_kv_attend_f16 = _bind("gemv_kv_attend_f16", _attend_args)
gemv_kv_attend_bf16 = _bind("gemv_kv_attend_bf16", _attend_args)

EXPORTED = ("gemv_status_string", "gemv_last_hip_error",
            "gemv_last_hip_error_string", "gemv_f32", "gemv_f16", "gemv_bf16",
            "gemv_batched_f16", "gemv_batched_bf16", "gemv_multi_f32",
            "gemv_multi_f16", "gemv_multi_bf16", "gemv_gate_up_silu_f32",
            "gemv_gate_up_silu_f16", "gemv_gate_up_silu_bf16",
            "gemv_splitk_workspace_size", "gemv_splitk_f32", "gemv_splitk_f16",
            "gemv_splitk_bf16", "gemv_splitk_noalloc", "gemv_q8_f32", "gemv_q8_f16", "gemv_q8_bf16",
            "gemv_q8_run_family", "gemv_plan_q8", "gemv_read_probe",
            "gemv_read_probe_variant", "gemv_plan",
            "gemv_plan_splitk", "gemv_run_family", "gemv_test_refused_launch",
            "gemv_fp8_quantise_f32", "gemv_fp8_quantise_f16", "gemv_fp8_quantise_bf16",
            "gemv_fp8_f32", "gemv_fp8_f16", "gemv_fp8_bf16", "gemv_kv_append_f32",
            "gemv_kv_append_f16", "gemv_kv_append_bf16", "gemv_kv_attend_workspace_size",
            "gemv_kv_attend_f16", "gemv_kv_attend_bf16")


class GemvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {gemv_status_string(status).decode()}"
        if status == GEMV_ERROR_LAUNCH_FAILURE:
            msg += f" ({gemv_last_hip_error_string().decode()})"
        super().__init__(msg)


def plan(dtype: str, M: int, K: int, lda: int | None = None, nvec: int = 1,
         A_addr: int = 0, X_addr: int = 0, family: int = FAMILY_AUTO) -> dict:
    """The mapping libgemv would launch (host-only; no GPU needed)."""
    out = GemvPlan()
    rc = gemv_plan(DTYPE_CODES[dtype], M, K, K if lda is None else lda, nvec,
                   A_addr, X_addr, family, ctypes.byref(out))
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, "gemv_plan")
    return out.as_dict()


def plan_splitk(dtype: str, M: int, K: int, lda: int | None = None, splits: int = 0,
                A_addr: int = 0, x_addr: int = 0) -> dict:
    """The mapping gemv_splitk_* would launch (host-only)."""
    out = GemvPlan()
    rc = gemv_plan_splitk(DTYPE_CODES[dtype], M, K, K if lda is None else lda, splits,
                          A_addr, x_addr, ctypes.byref(out))
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, "gemv_plan_splitk")
    return out.as_dict()


def plan_q8(xdtype: str, M: int, K: int, ldq: int | None = None, Q_addr: int = 0,
            x_addr: int = 0, family: int = FAMILY_AUTO) -> dict:
    """The mapping gemv_q8_* would launch for int8 weights and x of type
    ``xdtype`` (host-only)."""
    out = GemvPlan()
    rc = gemv_plan_q8(DTYPE_CODES[xdtype], M, K, K if ldq is None else ldq, Q_addr, x_addr,
                      family, ctypes.byref(out))
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, "gemv_plan_q8")
    return out.as_dict()


def splitk_workspace_size(dtype: str, M: int, K: int, splits: int = 0) -> int:
    """Workspace bytes gemv_splitk_* needs (0: a single slice, none needed)."""
    n = ctypes.c_size_t(0)
    rc = gemv_splitk_workspace_size(DTYPE_CODES[dtype], M, K, splits, ctypes.byref(n))
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, "gemv_splitk_workspace_size")
    return n.value


# ---------------------------------------------------------------------------
# tensor helpers
# ---------------------------------------------------------------------------

def _torch():
    import torch  # noqa: PLC0415 - torch only allocates memory and streams
    return torch


def _dtype_name(t) -> str:
    torch = _torch()
    names = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
    if t.dtype not in names:
        raise TypeError(f"unsupported dtype {t.dtype}; expected float32, float16 or bfloat16")
    return names[t.dtype]


def _stream_handle(stream=None) -> int:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _check_matrix(A):
    if A.dim() != 2:
        raise ValueError("A must be 2-D (M, K)")
    if not A.is_cuda:
        raise ValueError("A must be a device tensor")
    M, K = A.shape
    if K > 1 and A.stride(1) != 1:
        raise ValueError("A must have unit column stride")
    # with one row, or no columns, the row pitch is never used: pass K, the
    # tightest value (so 16-byte alignment depends only on the pointers)
    lda = A.stride(0) if (M > 1 and K > 0) else K
    if lda < K:
        raise ValueError("A's row stride is smaller than K")
    return M, K, lda


def _check_out(out, shape, device):
    torch = _torch()
    if out is None:
        return torch.empty(shape, dtype=torch.float32, device=device)
    if out.dtype != torch.float32 or tuple(out.shape) != tuple(shape) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous float32 tensor of shape {tuple(shape)}")
    if out.device != device:
        raise ValueError("out is on another device")
    return out


def _check_bias(bias, M, device):
    torch = _torch()
    if bias is None:
        return None
    if bias.dtype != torch.float32 or bias.dim() != 1 or bias.shape[0] != M or not bias.is_contiguous():
        raise ValueError("bias must be a contiguous float32 tensor of shape (M,)")
    if bias.device != device:
        raise ValueError("bias is on another device")
    return bias


def gemv(A, x, bias=None, out=None, *, family: int = FAMILY_AUTO, stream=None):
    """y = A @ x (+ bias) in fp32 on A's device; returns y (M,) float32."""
    M, K, lda = _check_matrix(A)
    dt = _dtype_name(A)
    if x.dtype != A.dtype or x.dim() != 1 or x.shape[0] != K or not x.is_contiguous():
        raise ValueError("x must be a contiguous (K,) tensor of A's dtype")
    if x.device != A.device:
        raise ValueError("x is on another device")
    bias = _check_bias(bias, M, A.device)
    y = _check_out(out, (M,), A.device)
    args = (A.data_ptr(), lda, x.data_ptr(),
            bias.data_ptr() if bias is not None else None, y.data_ptr(), M, K)
    if family == FAMILY_AUTO:
        fn = {"f32": gemv_f32, "f16": gemv_f16, "bf16": gemv_bf16}[dt]
        rc = fn(*args, _stream_handle(stream))
        where = fn.__name__
    else:
        rc = gemv_run_family(DTYPE_CODES[dt], family, args[0], lda, args[2],
                             args[3], args[4], M, K, 1, _stream_handle(stream))
        where = "gemv_run_family"
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, where)
    return y


def gemv_batched(A, X, bias=None, out=None, *, family: int = FAMILY_AUTO,
                 stream=None):
    """Y = A @ X (+ bias) for X of shape (nvec, K), 1 <= nvec <= 64, fp16 or
    bf16; returns Y of shape (nvec, M) float32 (column j = output for X[j])."""
    M, K, lda = _check_matrix(A)
    dt = _dtype_name(A)
    if X.dtype != A.dtype or X.dim() != 2 or X.shape[1] != K or not X.is_contiguous():
        raise ValueError("X must be a contiguous (nvec, K) tensor of A's dtype")
    if X.device != A.device:
        raise ValueError("X is on another device")
    nvec = X.shape[0]
    bias = _check_bias(bias, M, A.device)
    Y = _check_out(out, (nvec, M), A.device)
    bptr = bias.data_ptr() if bias is not None else None
    if family == FAMILY_AUTO:
        if dt == "f32":
            raise TypeError("the batched entry points take float16 or bfloat16")
        fn = {"f16": gemv_batched_f16, "bf16": gemv_batched_bf16}[dt]
        rc = fn(A.data_ptr(), lda, X.data_ptr(), bptr, Y.data_ptr(), M, K, nvec,
                _stream_handle(stream))
        where = fn.__name__
    else:
        rc = gemv_run_family(DTYPE_CODES[dt], family, A.data_ptr(), lda,
                             X.data_ptr(), bptr, Y.data_ptr(), M, K, nvec,
                             _stream_handle(stream))
        where = "gemv_run_family"
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, where)
    return Y


def gemv_splitk(A, x, bias=None, out=None, *, splits: int = 0, workspace=None, stream=None):
    """y = A @ x (+ bias) by split-K (for few, long rows); returns y (M,)
    float32.  ``workspace``: a device tensor of at least
    ``splitk_workspace_size(...)`` bytes, allocated here through torch when
    not given."""
    torch = _torch()
    M, K, lda = _check_matrix(A)
    dt = _dtype_name(A)
    if x.dtype != A.dtype or x.dim() != 1 or x.shape[0] != K or not x.is_contiguous():
        raise ValueError("x must be a contiguous (K,) tensor of A's dtype")
    if x.device != A.device:
        raise ValueError("x is on another device")
    bias = _check_bias(bias, M, A.device)
    y = _check_out(out, (M,), A.device)
    need = splitk_workspace_size(dt, M, K, splits)
    if workspace is None:
        workspace = torch.empty(max(need // 4, 1), dtype=torch.float32, device=A.device)
    if workspace.device != A.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on A's device")
    ws_bytes = workspace.numel() * workspace.element_size()
    fn = {"f32": gemv_splitk_f32, "f16": gemv_splitk_f16, "bf16": gemv_splitk_bf16}[dt]
    rc = fn(A.data_ptr(), lda, x.data_ptr(), bias.data_ptr() if bias is not None else None,
            y.data_ptr(), M, K, splits, workspace.data_ptr(), ws_bytes, _stream_handle(stream))
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, fn.__name__)
    return y


def gemv_q8(Q, scale, x, bias=None, out=None, *, family: int = FAMILY_AUTO, stream=None):
    """Weight-only int8: y = scale * (Q @ x) (+ bias) with Q int8 (M, K)
    (unit column stride, row stride ldq), scale float32 (M,), x (K,) float32,
    float16 or bfloat16; returns y (M,) float32."""
    torch = _torch()
    if Q.dtype != torch.int8:
        raise TypeError("Q must be int8")
    M, K, ldq = _check_matrix(Q)
    if x.dim() != 1 or x.shape[0] != K or not x.is_contiguous() or x.device != Q.device:
        raise ValueError("x must be a contiguous (K,) tensor on Q's device")
    dt = _dtype_name(x)
    if (scale.dtype != torch.float32 or scale.dim() != 1 or scale.shape[0] != M
            or not scale.is_contiguous() or scale.device != Q.device):
        raise ValueError("scale must be a contiguous float32 (M,) tensor on Q's device")
    bias = _check_bias(bias, M, Q.device)
    y = _check_out(out, (M,), Q.device)
    bptr = bias.data_ptr() if bias is not None else None
    if family == FAMILY_AUTO:
        fn = {"f32": gemv_q8_f32, "f16": gemv_q8_f16, "bf16": gemv_q8_bf16}[dt]
        rc = fn(Q.data_ptr(), ldq, scale.data_ptr(), x.data_ptr(), bptr, y.data_ptr(), M, K,
                _stream_handle(stream))
        where = fn.__name__
    else:
        rc = gemv_q8_run_family(DTYPE_CODES[dt], family, Q.data_ptr(), ldq, scale.data_ptr(),
                                x.data_ptr(), bptr, y.data_ptr(), M, K, _stream_handle(stream))
        where = "gemv_q8_run_family"
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, where)
    return y


def segment_table(segments) -> "ctypes.Array":
    """A gemv_segment_t array from (A_addr, lda, M, bias_addr_or_None, y_addr)
    tuples."""
    arr = (GemvSegment * len(segments))()
    for i, (A, lda, M, bias, y) in enumerate(segments):
        arr[i] = GemvSegment(A, lda, M, bias, y)
    return arr


def gemv_multi(As, x, biases=None, outs=None, *, stream=None):
    """y_i = A_i @ x (+ bias_i) for up to 8 matrices with the same K and dtype,
    in one launch; returns the list of y_i (float32)."""
    if not 1 <= len(As) <= MAX_SEGMENTS:
        raise ValueError(f"between 1 and {MAX_SEGMENTS} matrices")
    dt = _dtype_name(As[0])
    K = As[0].shape[1] if As[0].dim() == 2 else -1
    if x.dtype != As[0].dtype or x.dim() != 1 or x.shape[0] != K or not x.is_contiguous():
        raise ValueError("x must be a contiguous (K,) tensor of the matrices' dtype")
    biases = list(biases) if biases is not None else [None] * len(As)
    outs = list(outs) if outs is not None else [None] * len(As)
    segs, ys = [], []
    for A, b, o in zip(As, biases, outs):
        M, Ki, lda = _check_matrix(A)
        if A.dtype != As[0].dtype or Ki != K or A.device != x.device:
            raise ValueError("every matrix must have x's dtype, K and device")
        b = _check_bias(b, M, A.device)
        y = _check_out(o, (M,), A.device)
        ys.append(y)
        segs.append((A.data_ptr(), lda, M, b.data_ptr() if b is not None else None, y.data_ptr()))
    table = segment_table(segs)
    fn = {"f32": gemv_multi_f32, "f16": gemv_multi_f16, "bf16": gemv_multi_bf16}[dt]
    rc = fn(table, len(segs), x.data_ptr(), K, _stream_handle(stream))
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, fn.__name__)
    return ys


def gemv_gate_up_silu(A_gate, A_up, x, out=None, *, stream=None):
    """h = silu(A_gate @ x) * (A_up @ x) in one pass over both matrices
    (same shape, dtype and row stride); returns h (M,) float32."""
    M, K, lda = _check_matrix(A_gate)
    M2, K2, lda2 = _check_matrix(A_up)
    if (M2, K2) != (M, K) or A_up.dtype != A_gate.dtype or A_up.device != A_gate.device:
        raise ValueError("A_gate and A_up must have the same shape, dtype and device")
    if lda2 != lda and M > 1:
        raise ValueError("A_gate and A_up must have the same row stride")
    dt = _dtype_name(A_gate)
    if x.dtype != A_gate.dtype or x.dim() != 1 or x.shape[0] != K or not x.is_contiguous():
        raise ValueError("x must be a contiguous (K,) tensor of the matrices' dtype")
    h = _check_out(out, (M,), A_gate.device)
    fn = {"f32": gemv_gate_up_silu_f32, "f16": gemv_gate_up_silu_f16,
          "bf16": gemv_gate_up_silu_bf16}[dt]
    rc = fn(A_gate.data_ptr(), A_up.data_ptr(), lda, x.data_ptr(), h.data_ptr(), M, K,
            _stream_handle(stream))
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, fn.__name__)
    return h


# ---------------------------------------------------------------------------
# e4m3 with a scale per block of 128
# ---------------------------------------------------------------------------

# These helpers run between launches of a few microseconds: the checks are
# ordered so that the usual call (contiguous tensors on the current device)
# passes through few of them.
if _torch_runtime is not None:
    _F32, _I32 = _torch_runtime.float32, _torch_runtime.int32
    _E4M3_BYTES = (_torch_runtime.float8_e4m3fn, _torch_runtime.uint8)

    def _by_dtype(f32, f16, bf16):
        return {_torch_runtime.float32: f32, _torch_runtime.float16: f16, _torch_runtime.bfloat16: bf16}

    _QUANTISE = _by_dtype(gemv_fp8_quantise_f32, gemv_fp8_quantise_f16, gemv_fp8_quantise_bf16)
    _PRODUCT = _by_dtype(gemv_fp8_f32, gemv_fp8_f16, gemv_fp8_bf16)
    _APPEND = _by_dtype(gemv_kv_append_f32, gemv_kv_append_f16, gemv_kv_append_bf16)
    _KV_FORMATS = {_torch_runtime.int8: KV_INT8, _torch_runtime.float8_e4m3fn: KV_E4M3}
    _ATTEND = {_torch_runtime.float16: gemv_kv_attend_f16, _torch_runtime.bfloat16: gemv_kv_attend_bf16}


def _entry(table, dtype):
    fn = table.get(dtype)
    if fn is None:
        raise TypeError(f"unsupported dtype {dtype}; expected one of {', '.join(str(d) for d in table)}")
    return fn


def _call(dev, stream, fn, *args):
    """fn(*args, stream handle) with device ``dev`` current, on the given
    stream or the current one of that device; raises on a failure code."""
    torch = _torch_runtime
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, fn.__name__)


def _empty(near, shape, dtype, stream):
    """Memory on ``near``'s device for a call on ``stream`` (None: the current
    one): allocated there, so that whoever had it, or has it next, is ordered
    with the call."""
    if stream is None:
        return near.new_empty(shape, dtype=dtype)
    with _torch_runtime.cuda.stream(stream):
        return near.new_empty(shape, dtype=dtype)


def _rows(t, name, dev):
    """(rows, columns, row stride) of a matrix with unit column stride on
    device ``dev``."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    if dev < 0 or t.get_device() != dev:
        raise ValueError(f"{name} must be a device tensor, all on one device")
    rows, cols = shape
    if rows > _MOST or cols > _MOST:
        raise ValueError(f"{name} has more rows or columns than an int counts")
    if t.is_contiguous():
        return rows, cols, cols
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    # with one row, or no columns, the pitch is never used
    pitch = t.stride(0) if rows > 1 and cols > 0 else cols
    if not cols <= pitch <= _MOST:
        raise ValueError(f"{name}'s row stride is smaller than its rows, or more than an int counts")
    return rows, cols, pitch


def _scales(t, name, rows, cols, dev):
    have, across, pitch = _rows(t, name, dev)
    if have != rows or across != cols or t.dtype is not _F32:
        raise ValueError(f"{name} must be a float32 tensor of shape {(rows, cols)}")
    return pitch


def gemv_fp8_quantise(X, block_rows: int = 1, out=None, scale=None, *, stream=None):
    """(Q, scale): X (rows, K) in float32, float16 or bfloat16 (unit column
    stride) held in e4m3 with a float32 scale for every ``block_rows`` rows (1
    for activations, 128 for weights) and 128 columns.  Q is float8_e4m3fn
    (rows, K), scale (ceil(rows / block_rows), ceil(K / 128))."""
    if block_rows != 1 and block_rows != FP8_BLOCK:
        raise ValueError("block_rows must be 1 or 128")
    fn = _entry(_QUANTISE, X.dtype)
    dev = X.get_device()
    rows, K, ldx = _rows(X, "X", dev)
    lines, blocks = -(-rows // block_rows), (K + FP8_BLOCK - 1) // FP8_BLOCK
    if out is None:
        out = _empty(X, (rows, K), _torch_runtime.float8_e4m3fn, stream)
        ldq = K
    else:
        if out.dtype not in _E4M3_BYTES:
            raise TypeError("out must be float8_e4m3fn (or its bytes as uint8)")
        have, across, ldq = _rows(out, "out", dev)
        if (have, across) != (rows, K):
            raise ValueError("out must have X's shape")
    if scale is None:
        scale = _empty(X, (lines, blocks), _F32, stream)
        lds = blocks
    else:
        lds = _scales(scale, "scale", lines, blocks, dev)
    _call(dev, stream, fn, X.data_ptr(), ldx, out.data_ptr(), ldq, scale.data_ptr(), lds, rows, K, block_rows)
    return out, scale


def gemv_fp8(W, w_scale, X, x_scale, bias=None, out=None, *, out_dtype=None, stream=None):
    """Y (nvec, M) = X @ W.T (+ bias) for e4m3 W (M, K) with w_scale
    (ceil(M / 128), ceil(K / 128)) and e4m3 X (nvec, K) with x_scale (nvec,
    ceil(K / 128)), as ``gemv_fp8_quantise`` gives them; any nvec.  Y is float32,
    or ``out_dtype`` / out's dtype (float16, bfloat16); out may be a column
    slice of a wider matrix."""
    if W.dtype not in _E4M3_BYTES or X.dtype not in _E4M3_BYTES:
        raise TypeError("W and X must be float8_e4m3fn (or its bytes as uint8)")
    dev = W.get_device()
    M, K, ldw = _rows(W, "W", dev)
    nvec, Kx, ldx = _rows(X, "X", dev)
    if Kx != K:
        raise ValueError("W and X must have the same number of columns")
    blocks = (K + FP8_BLOCK - 1) // FP8_BLOCK
    ldws = _scales(w_scale, "w_scale", (M + FP8_BLOCK - 1) // FP8_BLOCK, blocks, dev)
    ldxs = _scales(x_scale, "x_scale", nvec, blocks, dev)
    if bias is not None:
        bias = _check_bias(bias, M, W.device).data_ptr()
    if out is None:
        if out_dtype is None:
            out_dtype = _F32
        fn = _entry(_PRODUCT, out_dtype)
        out = _empty(W, (nvec, M), out_dtype, stream)
        ldy = M
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out is not of out_dtype")
        fn = _entry(_PRODUCT, out.dtype)
        rows, cols, ldy = _rows(out, "out", dev)
        if (rows, cols) != (nvec, M):
            raise ValueError(f"out must be of shape {(nvec, M)}")
    _call(dev, stream, fn, W.data_ptr(), ldw, w_scale.data_ptr(), ldws, X.data_ptr(), ldx, x_scale.data_ptr(),
          ldxs, bias, out.data_ptr(), ldy, M, K, nvec)
    return out


# ---------------------------------------------------------------------------
# a paged key/value cache in 8 bits
# ---------------------------------------------------------------------------

class KVCache:
    """A paged key/value cache in int8 or e4m3 with a float32 scale per block
    of 16 tokens and head, over the caller's tensors:

    k (pages, heads, page_size, dim), v (pages, heads, page_size // 16, dim,
    16), both int8 or both float8_e4m3fn; k_scale and v_scale (pages, heads,
    page_size // 16) float32; all contiguous on one device.  ``KVCache.empty``
    allocates them."""

    def __init__(self, k, v, k_scale, v_scale):
        _torch()
        shape = k.shape
        if len(shape) != 4 or v.dim() != 5:
            raise ValueError("k must be (pages, heads, page_size, dim) and v (pages, heads, page_size // 16, dim, 16)")
        pages, heads, page_size, dim = shape
        if page_size not in (16, 32, 64, 128, 256) or dim not in (64, 128, 256):
            raise ValueError("page_size must be 16, 32, 64, 128 or 256 and dim 64, 128 or 256")
        blocks = page_size // KV_BLOCK
        if v.shape != (pages, heads, blocks, dim, KV_BLOCK):
            raise ValueError(f"v must be of shape {(pages, heads, blocks, dim, KV_BLOCK)}")
        cache_format = _KV_FORMATS.get(k.dtype)
        if cache_format is None or v.dtype is not k.dtype:
            raise TypeError("k and v must both be int8 or both float8_e4m3fn")
        scale = (pages, heads, blocks)
        if k_scale.dtype is not _F32 or v_scale.dtype is not _F32 or k_scale.shape != scale or v_scale.shape != scale:
            raise ValueError(f"k_scale and v_scale must be float32 tensors of shape {scale}")
        dev = k.get_device()
        if dev < 0 or not (dev == v.get_device() == k_scale.get_device() == v_scale.get_device()) or not (
                k.is_contiguous() and v.is_contiguous() and k_scale.is_contiguous() and v_scale.is_contiguous()):
            raise ValueError("the cache's tensors must be contiguous on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.dim = pages, heads, page_size, dim
        self._device = dev
        self._struct = KvCacheStruct(cache_format, pages, heads, page_size, dim, k.data_ptr(),
                                     v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())
        self._ref = ctypes.byref(self._struct)

    @classmethod
    def empty(cls, pages: int, heads: int, dim: int, *, page_size: int = 64, dtype=None, device="cuda"):
        """A cache in newly allocated memory (contents undefined); dtype int8
        (the default) or float8_e4m3fn."""
        torch = _torch()
        dtype = torch.int8 if dtype is None else dtype
        blocks = page_size // KV_BLOCK
        scale = (pages, heads, blocks)
        return cls(torch.empty((pages, heads, page_size, dim), dtype=dtype, device=device),
                   torch.empty((pages, heads, blocks, dim, KV_BLOCK), dtype=dtype, device=device),
                   torch.empty(scale, dtype=torch.float32, device=device),
                   torch.empty(scale, dtype=torch.float32, device=device))


def _kv_batch(cache, table, seq_lens, starts, rows):
    dev = cache._device
    shape = table.shape
    if len(shape) != 2 or table.dtype is not _I32:
        raise ValueError("table must be an int32 (sequences, pages) tensor")
    sequences, width = shape
    pitch = width
    if not table.is_contiguous():
        pitch = table.stride(0) if sequences > 1 else width
        if (width > 1 and table.stride(1) != 1) or not width <= pitch <= _MOST:
            raise ValueError("table must have unit column stride and a row stride of at least its width")
    if seq_lens.dtype is not _I32 or seq_lens.shape != (sequences,) or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous int32 (sequences,) tensor")
    if table.get_device() != dev or seq_lens.get_device() != dev:
        raise ValueError("table and seq_lens must be on the cache's device")
    if starts is None:
        if rows != sequences:
            raise ValueError("without starts every sequence has one row")
        return KvBatchStruct(sequences, table.data_ptr(), pitch, width, seq_lens.data_ptr(), None)
    if starts.dtype is not _I32 or starts.shape != (sequences + 1,) or not starts.is_contiguous():
        raise ValueError("starts must be a contiguous int32 (sequences + 1,) tensor")
    if starts.get_device() != dev:
        raise ValueError("starts must be on the cache's device")
    return KvBatchStruct(sequences, table.data_ptr(), pitch, width, seq_lens.data_ptr(), starts.data_ptr())


def _heads(t, name, cache):
    """(rows, heads, row stride) of a (rows, heads, dim) tensor whose rows may
    be columns of a wider matrix."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != cache.dim or t.get_device() != cache._device:
        raise ValueError(f"{name} must be (rows, heads, {cache.dim}) on the cache's device")
    rows, heads, dim = shape
    if t.is_contiguous():
        return rows, heads, heads * dim
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim):
        raise ValueError(f"{name}'s heads must lie one behind the other in a row")
    pitch = t.stride(0) if rows > 1 else heads * dim
    if not heads * dim <= pitch <= _MOST:
        raise ValueError(f"{name}'s row stride is smaller than its rows, or more than an int counts")
    return rows, heads, pitch


def gemv_kv_append(cache, K, V, table, seq_lens, starts=None, *, stream=None):
    """Write the new tokens' keys and values, K and V (rows, heads, dim) in
    float32, float16 or bfloat16, into the cache.

    table (sequences, pages) int32 names each sequence's pages, seq_lens
    (sequences,) int32 its length with the new tokens; its new tokens are the
    last ones, in rows starts[b] .. starts[b + 1] - 1 (starts (sequences + 1,)
    int32; None: one row for each sequence).  Rows behind the last start are
    ignored."""
    rows, heads, ldk = _heads(K, "K", cache)
    vrows, vheads, ldv = _heads(V, "V", cache)
    if heads != cache.heads or vheads != heads or vrows != rows or V.dtype is not K.dtype:
        raise ValueError("K and V must have the cache's heads, the same rows and the same dtype")
    fn = _entry(_APPEND, K.dtype)
    batch = _kv_batch(cache, table, seq_lens, starts, rows)
    _call(cache._device, stream, fn, cache._ref, K.data_ptr(), ldk, V.data_ptr(), ldv, rows, ctypes.byref(batch))


@functools.lru_cache(maxsize=256)
def _attend_workspace(q_heads, heads, dim, rows, sequences, one_each, table_width, page_size, window, sinks):
    n = ctypes.c_size_t(0)
    rc = gemv_kv_attend_workspace_size(q_heads, heads, dim, rows, sequences, one_each, table_width, page_size, window,
                                       sinks, ctypes.byref(n))
    if rc != GEMV_SUCCESS:
        raise GemvError(rc, "gemv_kv_attend_workspace_size")
    return n.value


def kv_attend_workspace_size(cache, q_heads: int, rows: int, sequences: int, table_width: int, *,
                             one_each: bool = True, window: int = 0, sinks: int = 0) -> int:
    """Workspace bytes that ``gemv_kv_attend`` needs (0: none); one_each: the
    call has no ``starts``.  It depends on these sizes only."""
    return _attend_workspace(q_heads, cache.heads, cache.dim, rows, sequences, int(one_each), table_width,
                             cache.page_size, window, sinks)


def gemv_kv_attend(Q, cache, table, seq_lens, starts=None, *, scale=None, window: int = 0, sinks: int = 0,
                   out=None, workspace=None, stream=None):
    """Causal attention of the batch's new tokens, Q (rows, q_heads, dim) in
    float16 or bfloat16, over the cache, which holds their own keys and values
    already; returns (rows, q_heads, dim) of Q's dtype.

    table, seq_lens and starts as for ``gemv_kv_append``.  scale: 1 / sqrt(dim)
    by default.  window > 0: a token sees the last ``window`` tokens (itself
    among them) and the first ``sinks``.  Rows of out behind the last start are
    left as they were.  workspace: a device tensor of at least
    ``kv_attend_workspace_size(...)`` bytes, allocated here through torch when
    not given."""
    fn = _entry(_ATTEND, Q.dtype)
    if not (-_MOST <= window <= _MOST and -_MOST <= sinks <= _MOST):
        raise ValueError("window and sinks must be what an int holds")
    rows, q_heads, ldq = _heads(Q, "Q", cache)
    if out is None:
        out = _empty(Q, (rows, q_heads, cache.dim), Q.dtype, stream)
        ldo = q_heads * cache.dim
    else:
        if out.dtype is not Q.dtype or out.shape != Q.shape:
            raise ValueError("out must have Q's shape and dtype")
        ldo = _heads(out, "out", cache)[2]
    batch = _kv_batch(cache, table, seq_lens, starts, rows)
    need = _attend_workspace(q_heads, cache.heads, cache.dim, rows, batch.sequences, starts is None,
                             batch.table_width, cache.page_size, window, sinks)
    if workspace is not None:
        if workspace.get_device() != cache._device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the cache's device")
        need = workspace.numel() * workspace.element_size()
    elif need:
        workspace = _empty(Q, need // 4, _F32, stream)
    _call(cache._device, stream, fn, cache._ref, Q.data_ptr(), ldq, out.data_ptr(), ldo, q_heads, rows,
          ctypes.byref(batch), cache.dim ** -0.5 if scale is None else scale, window, sinks,
          workspace.data_ptr() if workspace is not None else None, need)
    return out
