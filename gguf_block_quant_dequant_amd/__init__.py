"""Python binding of libgguf_qk (include/gguf_qk.h, gguf_kv.h, gguf_tokens.h,
gguf_file.h): GGUF Q8_0 / Q4_K dequant, fused dequant x activation products, and
the steps around them (rotation of queries and keys, paged key-value cache,
attention of one or several new tokens, log probabilities, verification of drafted
tokens) on an MI355X (gfx950).

Argument marshalling only: each function takes torch device tensors, passes
their raw pointers, sizes and the current HIP stream to the C entry point of
the same name, and raises on a negative status. Every arithmetic step runs in
the library's kernels; there is no CPU path. If the library has not been built
the first call raises.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct
from typing import NamedTuple, Optional

import torch

from .build import LIB_PATH, TIMELINE_LIB_PATH

TYPE_Q8_0 = 8
TYPE_Q4_K = 12
TYPE_Q4_0 = 2
TYPE_Q6_K = 14

OK = 0
ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ALIAS, ERR_DEVICE, ERR_LAUNCH, ERR_LIMIT = -1, -2, -3, -4, -5, -6, -7
ERR_FORMAT, ERR_IO, ERR_NOT_FOUND = -8, -9, -10

# GGUF tensor and metadata value type ids (include/gguf_file.h)
TENSOR_F32, TENSOR_F16, TENSOR_Q4_0, TENSOR_Q8_0, TENSOR_Q4_K, TENSOR_Q6_K, TENSOR_BF16 = 0, 1, 2, 8, 12, 14, 30
(VALUE_U8, VALUE_I8, VALUE_U16, VALUE_I16, VALUE_U32, VALUE_I32, VALUE_F32, VALUE_BOOL, VALUE_STRING,
 VALUE_ARRAY, VALUE_U64, VALUE_I64, VALUE_F64) = range(13)
_SCALAR_FMT = {VALUE_U8: "<B", VALUE_I8: "<b", VALUE_U16: "<H", VALUE_I16: "<h", VALUE_U32: "<I",
               VALUE_I32: "<i", VALUE_F32: "<f", VALUE_BOOL: "<?", VALUE_U64: "<Q", VALUE_I64: "<q",
               VALUE_F64: "<d"}

_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SIGS = {
    "gguf_qk_abi_version": (ctypes.c_int, []),
    "gguf_qk_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "gguf_row_bytes": (_I64, [ctypes.c_int, _I64]),
    "dequant_q8_0": (ctypes.c_int, [_P, _P, _I64, _I64, _P]),
    "dequant_q4_k": (ctypes.c_int, [_P, _P, _I64, _I64, _P]),
    "dequant_q4_k_bf16": (ctypes.c_int, [_P, _P, _I64, _I64, _P]),
    "gguf_qmatvec_q8_0": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _P]),
    "gguf_qmatvec_q4_k": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _P]),
    "dequant_q4_0": (ctypes.c_int, [_P, _P, _I64, _I64, _P]),
    "dequant_q6_k": (ctypes.c_int, [_P, _P, _I64, _I64, _P]),
    "gguf_qmatvec_q4_0": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _P]),
    "gguf_qmatvec_q6_k": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _P]),
    "gguf_qmatmul_q4_k": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _P]),
    "gguf_qmatmul_q4_k_multi": (ctypes.c_int, [_P, _P, _P, ctypes.c_int32, _P, _I64, _I64, _P]),
    "gguf_qmatmul_f32_q8_0": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _P]),
    "gguf_qmatmul_f32_q4_k": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _P]),
    "gguf_qmatmul_f32_q8_0_multi": (ctypes.c_int, [_P, _P, _P, ctypes.c_int32, _P, _I64, _I64, _P]),
    "gguf_qmatmul_f32_q4_k_multi": (ctypes.c_int, [_P, _P, _P, ctypes.c_int32, _P, _I64, _I64, _P]),
    "gguf_qk_probe_read": (ctypes.c_int, [_P, _I64, _P, _P]),
    "gguf_qk_probe_latency": (ctypes.c_int, [_P, _I64, _I64, _P, _P]),
    "gguf_qk_stream_release": (ctypes.c_int, [_P]),
    "gguf_qk_last_launch": (ctypes.c_int, []),
    "gguf_qk_timeline_setup": (ctypes.c_int, [ctypes.c_uint64]),
    "gguf_qk_timeline_fetch": (ctypes.c_int, [_P, _I64]),
    "gguf_qmatvec_batch": (ctypes.c_int, [_P, ctypes.c_int32, _P]),
    "gguf_qmatvec_batch_ep": (ctypes.c_int, [_P, _P, ctypes.c_int32, _P]),
    "gguf_rmsnorm_prep_f32": (ctypes.c_int, [_P, _P, _P, _P, _I64, _P]),
    "gguf_rmsnorm_f32": (ctypes.c_int, [_P, _P, ctypes.c_float, _P, _I64, _P]),
    "gguf_swiglu_f32": (ctypes.c_int, [_P, _P, _P, _I64, _P]),
    "gguf_add_f32": (ctypes.c_int, [_P, _P, _P, _I64, _P]),
    "gguf_kv_page_bytes": (_I64, [ctypes.c_int, _I64, _I64, _I64]),
    "gguf_kv_append": (ctypes.c_int, [_P, _P, _P, ctypes.c_int32, _I64, _I64, _P, _P, _P, _P, _I64, _I64, _P]),
    "gguf_attn_decode_workspace": (_I64, [_P, _I64, _I64, _I64, ctypes.c_int32]),
    "gguf_attn_decode": (ctypes.c_int, [_P, _P, _I64, _P, _I64, _I64, _I64, _P, _I64, _P, _I64, ctypes.c_float,
                                        _I64, ctypes.c_int32, _P, _I64, _P]),
    "gguf_kv_evict_workspace": (_I64, [_P, _I64, _I64, _I64]),
    "gguf_kv_evict": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _I64, _I64, _I64, _P, _I64, _P]),
    "gguf_logprobs_workspace": (_I64, [_I64, _I64, ctypes.c_int32]),
    "gguf_logprobs": (ctypes.c_int, [_P, ctypes.c_int32, _I64, _I64, _I64, _P, _I64, ctypes.c_int32, _P, _P, _P,
                                     _P, _P, _I64, _P]),
    "gguf_qk_rope": (ctypes.c_int, [_P, _I64, _P, _I64, _I64, _P, _I64, _P, _I64, _I64, ctypes.c_int32, _I64, _I64, _P,
                                    _P, ctypes.c_float, _P, _P]),
    "gguf_attn_extend_workspace": (_I64, [_P, ctypes.c_int32, _I64, _I64, _I64, _I64, _I64, _I64]),
    "gguf_attn_extend": (ctypes.c_int, [_P, _P, ctypes.c_int32, _I64, _P, _I64, _P, _I64, _I64, _I64, _P, _I64, _P, _I64,
                                        ctypes.c_float, _I64, _I64, _P, _I64, _P]),
    "gguf_verify_draft_workspace": (_I64, [_I64, _I64, _I64, ctypes.c_int32]),
    "gguf_verify_draft": (ctypes.c_int, [_P, _I64, _P, _I64, ctypes.c_int32, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P,
                                         _P, _P, _P, _I64, _P]),
    "gguf_tensor_nbytes": (_I64, [ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_int64)]),
    "gguf_file_open": (ctypes.c_int, [ctypes.c_char_p, ctypes.POINTER(ctypes.c_void_p)]),
    "gguf_file_close": (None, [_P]),
    "gguf_file_version": (ctypes.c_int32, [_P]),
    "gguf_file_tensor_count": (_I64, [_P]),
    "gguf_file_kv_count": (_I64, [_P]),
    "gguf_file_alignment": (_I64, [_P]),
    "gguf_file_data_offset": (_I64, [_P]),
    "gguf_file_size": (_I64, [_P]),
    "gguf_file_tensor": (ctypes.c_int, [_P, _I64, _P]),
    "gguf_file_kv": (ctypes.c_int, [_P, _I64, _P]),
    "gguf_file_find_tensor": (_I64, [_P, ctypes.c_char_p]),
    "gguf_file_find_kv": (_I64, [_P, ctypes.c_char_p]),
    "gguf_file_kv_array_string": (ctypes.c_int, [_P, _I64, _I64, ctypes.POINTER(ctypes.c_void_p),
                                                 ctypes.POINTER(ctypes.c_int64)]),
    "gguf_file_upload_tensor": (ctypes.c_int, [_P, _I64, _P, _P]),
}


class GgufTensorInfo(ctypes.Structure):
    """struct gguf_tensor_info of the C ABI."""
    _fields_ = [("name", ctypes.c_char_p), ("type", ctypes.c_int32), ("n_dims", ctypes.c_int32),
                ("dims", ctypes.c_int64 * 4), ("offset", ctypes.c_int64), ("nbytes", ctypes.c_int64),
                ("data", ctypes.c_void_p)]


class GgufKvInfo(ctypes.Structure):
    """struct gguf_kv_info of the C ABI."""
    _fields_ = [("key", ctypes.c_char_p), ("type", ctypes.c_int32), ("elem_type", ctypes.c_int32),
                ("count", ctypes.c_int64), ("data", ctypes.c_void_p), ("nbytes", ctypes.c_int64)]


class GemvEntry(ctypes.Structure):
    """struct gguf_qk_gemv of the C ABI."""
    _fields_ = [("W", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("type", ctypes.c_int32),
                ("stage", ctypes.c_int32), ("reserved", ctypes.c_int32 * 2)]


def library_path() -> str:
    """The build of libgguf_qk.so that lib() loads: GGUF_QK_LIBRARY=<path> (another
    build of the same library: the sanitized host build, measurement of build
    variants), else with GGUF_QK_TIMELINE=1 the instrumented build (stage
    timelines), else the default build."""
    path = TIMELINE_LIB_PATH if os.environ.get("GGUF_QK_TIMELINE") == "1" else LIB_PATH
    return os.environ.get("GGUF_QK_LIBRARY", path)


def lib() -> ctypes.CDLL:
    """The loaded libgguf_qk.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m gguf_block_quant_dequant_amd.build`")
        L = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


class GgufQkError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gguf_qk_strerror(status)} (status {status})")


class GgufQkArgumentError(GgufQkError, ValueError):
    pass


def _check(status: int, where: str) -> None:
    if status == OK:
        return
    if status in (ERR_DEVICE, ERR_LAUNCH):
        raise GgufQkError(status, where)
    raise GgufQkArgumentError(status, where)


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _rows_cols(W: torch.Tensor, fmt: int, rows, cols):
    if rows is None or cols is None:
        if W.dim() != 2:
            raise ValueError("pass rows and cols, or W as a [rows, row_bytes] uint8 tensor")
        r = W.shape[0]
        rb = W.shape[1]
        blk_b, blk_w = {TYPE_Q8_0: (34, 32), TYPE_Q4_K: (144, 256), TYPE_Q4_0: (18, 32),
                        TYPE_Q6_K: (210, 256)}[fmt]
        if rb % blk_b:
            raise ValueError("W row bytes are not a whole number of blocks")
        rows = r if rows is None else rows
        cols = rb // blk_b * blk_w if cols is None else cols
    need = gguf_row_bytes(fmt, cols)
    if need < 0:
        raise GgufQkArgumentError(need, "row bytes")
    if W.numel() * W.element_size() < rows * need:
        raise ValueError("W is smaller than rows x row bytes")
    return int(rows), int(cols)


def gguf_qk_abi_version() -> int:
    return lib().gguf_qk_abi_version()


def gguf_qk_strerror(status: int) -> str:
    return lib().gguf_qk_strerror(status).decode()


def gguf_row_bytes(type_id: int, cols: int) -> int:
    return lib().gguf_row_bytes(type_id, cols)


def _dequant(name, fmt, W, out, rows, cols, out_dtype, stream):
    rows, cols = _rows_cols(W, fmt, rows, cols)
    if out is None:
        out = torch.empty((rows, cols), dtype=out_dtype, device=W.device)
    if out.numel() < rows * cols:
        raise ValueError("out is too small")
    _check(getattr(lib(), name)(_dev(W, "W", torch.uint8), _dev(out, "out", out_dtype), rows, cols,
                                _stream(stream)), name)
    return out


def dequant_q8_0(W, out=None, rows=None, cols=None, stream=None):
    """fp32 [rows, cols] dequant of a Q8_0 matrix (bit-exact)."""
    return _dequant("dequant_q8_0", TYPE_Q8_0, W, out, rows, cols, torch.float32, stream)


def dequant_q4_k(W, out=None, rows=None, cols=None, stream=None):
    """fp32 [rows, cols] dequant of a Q4_K matrix (bit-exact)."""
    return _dequant("dequant_q4_k", TYPE_Q4_K, W, out, rows, cols, torch.float32, stream)


def dequant_q4_0(W, out=None, rows=None, cols=None, stream=None):
    """fp32 [rows, cols] dequant of a Q4_0 matrix (bit-exact)."""
    return _dequant("dequant_q4_0", TYPE_Q4_0, W, out, rows, cols, torch.float32, stream)


def dequant_q6_k(W, out=None, rows=None, cols=None, stream=None):
    """fp32 [rows, cols] dequant of a Q6_K matrix (bit-exact)."""
    return _dequant("dequant_q6_k", TYPE_Q6_K, W, out, rows, cols, torch.float32, stream)


def dequant_q4_k_bf16(W, out=None, rows=None, cols=None, stream=None):
    """bf16 [rows, cols]: the fp32 dequant rounded to nearest-even."""
    return _dequant("dequant_q4_k_bf16", TYPE_Q4_K, W, out, rows, cols, torch.bfloat16, stream)


def _matvec(name, fmt, W, x, y, rows, cols, stream):
    rows, cols = _rows_cols(W, fmt, rows, x.numel() if cols is None else cols)
    if x.numel() != cols:
        raise ValueError(f"x has {x.numel()} elements, expected {cols}")
    if y is None:
        y = torch.empty(rows, dtype=torch.float32, device=W.device)
    if y.numel() != rows:
        raise ValueError(f"y has {y.numel()} elements, expected {rows}")
    _check(getattr(lib(), name)(_dev(W, "W", torch.uint8), _dev(x, "x", torch.float32),
                                _dev(y, "y", torch.float32), rows, cols, _stream(stream)), name)
    return y


def gguf_qmatvec_q8_0(W, x, y=None, rows=None, cols=None, stream=None):
    """y = dequant(W) @ x for a Q8_0 W (fp32 x and y)."""
    return _matvec("gguf_qmatvec_q8_0", TYPE_Q8_0, W, x, y, rows, cols, stream)


def gguf_qmatvec_q4_k(W, x, y=None, rows=None, cols=None, stream=None):
    """y = dequant(W) @ x for a Q4_K W (fp32 x and y)."""
    return _matvec("gguf_qmatvec_q4_k", TYPE_Q4_K, W, x, y, rows, cols, stream)


def gguf_qmatvec_q4_0(W, x, y=None, rows=None, cols=None, stream=None):
    """y = dequant(W) @ x for a Q4_0 W (fp32 x and y)."""
    return _matvec("gguf_qmatvec_q4_0", TYPE_Q4_0, W, x, y, rows, cols, stream)


def gguf_qmatvec_q6_k(W, x, y=None, rows=None, cols=None, stream=None):
    """y = dequant(W) @ x for a Q6_K W (fp32 x and y)."""
    return _matvec("gguf_qmatvec_q6_k", TYPE_Q6_K, W, x, y, rows, cols, stream)


def gguf_qmatmul_q4_k(W, X, Y=None, rows=None, stream=None):
    """Y = X @ dequant(W)^T for a Q4_K W, X bf16 [n_tokens, cols], Y bf16 [n_tokens, rows]."""
    if X.dim() != 2:
        raise ValueError("X must be [n_tokens, cols]")
    n, cols = X.shape
    rows, cols = _rows_cols(W, TYPE_Q4_K, rows, cols)
    if Y is None:
        Y = torch.empty((n, rows), dtype=torch.bfloat16, device=W.device)
    if Y.numel() != n * rows:
        raise ValueError("Y must have n_tokens x rows elements")
    _check(lib().gguf_qmatmul_q4_k(_dev(W, "W", torch.uint8), _dev(X, "X", torch.bfloat16),
                                   _dev(Y, "Y", torch.bfloat16), n, rows, cols, _stream(stream)),
           "gguf_qmatmul_q4_k")
    return Y


def gguf_qmatmul_q4_k_multi(Ws, X, Ys=None, rows=None, stream=None):
    """Y[m] = X @ dequant(Ws[m])^T for up to four Q4_K matrices of one X (same
    cols), one launch; returns the list of Y (bf16 [n_tokens, rows[m]])."""
    if X.dim() != 2:
        raise ValueError("X must be [n_tokens, cols]")
    if not 1 <= len(Ws) <= 4:
        raise ValueError("one to four matrices")
    n, cols = X.shape
    rows = list(rows) if rows is not None else [None] * len(Ws)
    if len(rows) != len(Ws):
        raise ValueError("one row count per matrix")
    rows = [_rows_cols(W, TYPE_Q4_K, r, cols)[0] for W, r in zip(Ws, rows)]
    if Ys is None:
        Ys = [torch.empty((n, r), dtype=torch.bfloat16, device=X.device) for r in rows]
    if len(Ys) != len(Ws) or any(Y.numel() != n * r for Y, r in zip(Ys, rows)):
        raise ValueError("one Y of n_tokens x rows[m] elements per matrix")
    k = len(Ws)
    warr = (ctypes.c_void_p * k)(*[_dev(W, "W", torch.uint8) for W in Ws])
    yarr = (ctypes.c_void_p * k)(*[_dev(Y, "Y", torch.bfloat16) for Y in Ys])
    rarr = (ctypes.c_int64 * k)(*rows)
    _check(lib().gguf_qmatmul_q4_k_multi(warr, yarr, rarr, k, _dev(X, "X", torch.bfloat16), n, cols,
                                         _stream(stream)),
           "gguf_qmatmul_q4_k_multi")
    return Ys


def _matmul_f32_multi(name, fmt, Ws, X, Ys, rows, stream):
    if X.dim() != 2:
        raise ValueError("X must be [n_tokens, cols]")
    if not 1 <= len(Ws) <= 4:
        raise ValueError("one to four matrices")
    n, cols = X.shape
    rows = list(rows) if rows is not None else [None] * len(Ws)
    if len(rows) != len(Ws):
        raise ValueError("one row count per matrix")
    rows = [_rows_cols(W, fmt, r, cols)[0] for W, r in zip(Ws, rows)]
    if Ys is None:
        Ys = [torch.empty((n, r), dtype=torch.float32, device=X.device) for r in rows]
    if len(Ys) != len(Ws) or any(Y.numel() != n * r for Y, r in zip(Ys, rows)):
        raise ValueError("one Y of n_tokens x rows[m] elements per matrix")
    k = len(Ws)
    warr = (ctypes.c_void_p * k)(*[_dev(W, "W", torch.uint8) for W in Ws])
    yarr = (ctypes.c_void_p * k)(*[_dev(Y, "Y", torch.float32) for Y in Ys])
    rarr = (ctypes.c_int64 * k)(*rows)
    _check(getattr(lib(), name)(warr, yarr, rarr, k, _dev(X, "X", torch.float32), n, cols, _stream(stream)),
           name)
    return Ys


def gguf_qmatmul_f32_q8_0_multi(Ws, X, Ys=None, rows=None, stream=None):
    """Y[m] = X @ dequant(Ws[m])^T for up to four Q8_0 matrices of one fp32 X, one launch."""
    return _matmul_f32_multi("gguf_qmatmul_f32_q8_0_multi", TYPE_Q8_0, Ws, X, Ys, rows, stream)


def gguf_qmatmul_f32_q4_k_multi(Ws, X, Ys=None, rows=None, stream=None):
    """Y[m] = X @ dequant(Ws[m])^T for up to four Q4_K matrices of one fp32 X, one launch."""
    return _matmul_f32_multi("gguf_qmatmul_f32_q4_k_multi", TYPE_Q4_K, Ws, X, Ys, rows, stream)


def _matmul_f32(name, fmt, W, X, Y, rows, stream):
    if X.dim() != 2:
        raise ValueError("X must be [n_tokens, cols]")
    n, cols = X.shape
    rows, cols = _rows_cols(W, fmt, rows, cols)
    if Y is None:
        Y = torch.empty((n, rows), dtype=torch.float32, device=W.device)
    if Y.numel() != n * rows:
        raise ValueError("Y must have n_tokens x rows elements")
    _check(getattr(lib(), name)(_dev(W, "W", torch.uint8), _dev(X, "X", torch.float32),
                                _dev(Y, "Y", torch.float32), n, rows, cols, _stream(stream)), name)
    return Y


def gguf_qmatmul_f32_q8_0(W, X, Y=None, rows=None, stream=None):
    """Y = X @ dequant(W)^T for a Q8_0 W, X fp32 [n_tokens, cols], Y fp32 [n_tokens, rows]."""
    return _matmul_f32("gguf_qmatmul_f32_q8_0", TYPE_Q8_0, W, X, Y, rows, stream)


def gguf_qmatmul_f32_q4_k(W, X, Y=None, rows=None, stream=None):
    """Y = X @ dequant(W)^T for a Q4_K W, X fp32 [n_tokens, cols], Y fp32 [n_tokens, rows]."""
    return _matmul_f32("gguf_qmatmul_f32_q4_k", TYPE_Q4_K, W, X, Y, rows, stream)


def gguf_qk_probe_read(buf, sink=None, stream=None):
    """Enqueue one streaming read of the whole device tensor `buf` (its byte size
    must be a multiple of 16). Returns the 16-byte-aligned sink tensor."""
    nbytes = buf.numel() * buf.element_size()
    if sink is None:
        sink = torch.zeros(4, dtype=torch.int32, device=buf.device)
    _check(lib().gguf_qk_probe_read(_dev(buf, "buf"), nbytes, _dev(sink, "sink", torch.int32),
                                    _stream(stream)), "gguf_qk_probe_read")
    return sink


def gguf_qk_probe_latency(next_idx, steps, out=None, stream=None):
    """Enqueue the dependent-load chase over the int32 device tensor `next_idx`
    (a power-of-two number of entries); returns the int64 tensor out whose
    element 0 becomes the elapsed 100 MHz ticks of `steps` dependent loads."""
    if next_idx.dtype != torch.int32:
        raise TypeError("next_idx must be int32")
    if out is None:
        out = torch.zeros(2, dtype=torch.int64, device=next_idx.device)
    _check(lib().gguf_qk_probe_latency(_dev(next_idx, "next_idx", torch.int32), next_idx.numel(), int(steps),
                                       _dev(out, "out", torch.int64), _stream(stream)), "gguf_qk_probe_latency")
    return out


STREAM_SLOTS = 8   # GGUF_QK_STREAM_SLOTS: scratch slots per device
# GGUF_QK_LAUNCH_*: kernel families reported by gguf_qk_last_launch
(LAUNCH_NONE, LAUNCH_LK_SINGLE, LAUNCH_LK_TWO, LAUNCH_LK_THREE, LAUNCH_LK_GROUP, LAUNCH_LK_LONG, LAUNCH_LKS,
 LAUNCH_SPLIT_K, LAUNCH_OTHER, LAUNCH_ROWWISE) = range(10)


def gguf_qk_last_launch() -> int:
    """Kernel family (LAUNCH_*) of this thread's most recent GEMV launch."""
    return lib().gguf_qk_last_launch()


def gguf_qk_stream_release(stream=None):
    """Give back the scratch slot `stream` holds (synchronize the stream first)."""
    _check(lib().gguf_qk_stream_release(_stream(stream)), "gguf_qk_stream_release")


TIMELINE_SLOTS, TIMELINE_WAVES, TIMELINE_REC_BYTES = 4096, 2048, 32


def timeline_slot(key: int, mult: int) -> int:
    """Record slot of a launch key (its first weight pointer) under `mult`."""
    return ((key * mult) & ((1 << 64) - 1)) >> 52


def gguf_qk_timeline_setup(keys, seed=1):
    """Arm the instrumented build's per-wave stage records; picks an odd
    multiplier under which the launch keys `keys` take distinct slots and
    returns {key: slot}."""
    import random
    ks = sorted(set(int(k) for k in keys))
    rnd = random.Random(seed)
    for _ in range(100000):
        mult = rnd.getrandbits(64) | 1
        slots = [timeline_slot(k, mult) for k in ks]
        if len(set(slots)) == len(slots):
            _check(lib().gguf_qk_timeline_setup(mult), "gguf_qk_timeline_setup")
            return dict(zip(ks, slots))
    raise GgufQkError(ERR_LIMIT, "gguf_qk_timeline_setup: no multiplier separates the keys")


def gguf_qk_timeline_fetch():
    """The record array as a numpy uint32 array [4096, 2048, 8] (six time stamps,
    HW_ID, XCD id per wave)."""
    import numpy as np
    out = np.zeros((TIMELINE_SLOTS, TIMELINE_WAVES, TIMELINE_REC_BYTES // 4), dtype=np.uint32)
    _check(lib().gguf_qk_timeline_fetch(out.ctypes.data, out.nbytes), "gguf_qk_timeline_fetch")
    return out


class GemvEpEntry(ctypes.Structure):
    """struct gguf_qk_gemv_ep of the C ABI."""
    _fields_ = [("scale_ss", ctypes.c_void_p), ("scale_n", ctypes.c_int64), ("eps", ctypes.c_float),
                ("pair", ctypes.c_int32), ("residual", ctypes.c_void_p), ("norm_w", ctypes.c_void_p),
                ("norm_out", ctypes.c_void_p), ("ss_out", ctypes.c_void_p), ("act", ctypes.c_void_p),
                ("scale_v", ctypes.c_void_p)]


def _opt(t, name):
    return None if t is None else _dev(t, name, torch.float32)


class GemvBatch:
    """A prepared gguf_qmatvec_batch list: entries (type, W, x, y, stage) with
    device tensors; keeps the tensors alive and the C array built once.

    `epilogues` (optional, one per entry, None for none) are dicts with the
    gguf_qk_gemv_ep fields as keys (scale_ss, eps, pair, residual, norm_w,
    norm_out, ss_out, act, scale_v; tensors for the vectors); the batch then
    runs through gguf_qmatvec_batch_ep."""

    # floats each epilogue vector holds at least, for an entry of `rows` rows
    # (the C ABI takes these pointers without lengths)
    _EP_SIZES = {"residual": lambda r: r, "norm_w": lambda r: r, "norm_out": lambda r: r,
                 "act": lambda r: r, "ss_out": lambda r: (r + 63) // 64}

    def __init__(self, entries, epilogues=None):
        if epilogues is not None:
            if len(epilogues) != len(entries):
                raise ValueError("one epilogue (or None) per entry")
            for (_, _, x, y, _), e in zip(entries, epilogues):
                for key, need in self._EP_SIZES.items():
                    t = (e or {}).get(key)
                    if t is not None and t.numel() < need(y.numel()):
                        raise ValueError(f"epilogue {key} holds {t.numel()} floats, the entry needs "
                                         f"{need(y.numel())}")
                v = (e or {}).get("scale_v")
                if v is not None and v.numel() < x.numel():
                    raise ValueError(f"epilogue scale_v holds {v.numel()} floats, the entry needs {x.numel()}")
        self._keep = []
        arr = (GemvEntry * len(entries))()
        for i, (type_id, W, x, y, stage) in enumerate(entries):
            rows, cols = y.numel(), x.numel()
            _rows_cols(W, type_id, rows, cols)
            arr[i] = GemvEntry(_dev(W, "W", torch.uint8), _dev(x, "x", torch.float32),
                               _dev(y, "y", torch.float32), rows, cols, type_id, stage, (0, 0))
            self._keep.append((W, x, y))
        self.array = arr
        self.n = len(entries)
        self.ep = None
        if epilogues is not None:
            ep = (GemvEpEntry * len(entries))()
            for i, e in enumerate(epilogues):
                if not e:
                    continue
                ss = e.get("scale_ss")
                ep[i] = GemvEpEntry(_opt(ss, "scale_ss"), 0 if ss is None else ss.numel(),
                                    float(e.get("eps", 0.0)), int(e.get("pair", 0)),
                                    _opt(e.get("residual"), "residual"), _opt(e.get("norm_w"), "norm_w"),
                                    _opt(e.get("norm_out"), "norm_out"), _opt(e.get("ss_out"), "ss_out"),
                                    _opt(e.get("act"), "act"), _opt(e.get("scale_v"), "scale_v"))
                self._keep.append(tuple(v for v in e.values() if isinstance(v, torch.Tensor)))
            self.ep = ep


def gguf_qmatvec_batch(batch: GemvBatch, stream=None):
    """Run a prepared GemvBatch (steps in order on the stream)."""
    if batch.ep is not None:
        return gguf_qmatvec_batch_ep(batch, stream)
    _check(lib().gguf_qmatvec_batch(ctypes.cast(batch.array, ctypes.c_void_p), batch.n,
                                    _stream(stream)), "gguf_qmatvec_batch")


def gguf_qmatvec_batch_ep(batch: GemvBatch, stream=None):
    """Run a prepared GemvBatch with its per-entry epilogues."""
    ep = ctypes.cast(batch.ep, ctypes.c_void_p) if batch.ep is not None else None
    _check(lib().gguf_qmatvec_batch_ep(ctypes.cast(batch.array, ctypes.c_void_p), ep, batch.n,
                                       _stream(stream)), "gguf_qmatvec_batch_ep")


def _vec(t, name, n=None):
    p = _dev(t, name, torch.float32)
    if n is not None and t.numel() < n:
        raise ValueError(f"{name} is too small")
    return p


def gguf_rmsnorm_prep_f32(v, norm_w, vw=None, ss=None, stream=None):
    """vw = v * norm_w and ss[j] = sum of v^2 over elements 64 j .. 64 j + 63."""
    n = v.numel()
    vw = torch.empty_like(v) if vw is None else vw
    ss = torch.empty((n + 63) // 64, dtype=torch.float32, device=v.device) if ss is None else ss
    _check(lib().gguf_rmsnorm_prep_f32(_vec(v, "v"), _vec(norm_w, "norm_w", n), _vec(vw, "vw", n),
                                       _vec(ss, "ss", (n + 63) // 64), n, _stream(stream)),
           "gguf_rmsnorm_prep_f32")
    return vw, ss


def gguf_rmsnorm_f32(v, norm_w, eps, out=None, stream=None):
    """out = norm_w * v / sqrt(mean(v^2) + eps)."""
    n = v.numel()
    out = torch.empty_like(v) if out is None else out
    _check(lib().gguf_rmsnorm_f32(_vec(v, "v"), _vec(norm_w, "norm_w", n), float(eps),
                                  _vec(out, "out", n), n, _stream(stream)), "gguf_rmsnorm_f32")
    return out


def gguf_swiglu_f32(g, u, out=None, stream=None):
    """out = SiLU(g) * u."""
    n = g.numel()
    out = torch.empty_like(g) if out is None else out
    _check(lib().gguf_swiglu_f32(_vec(g, "g"), _vec(u, "u", n), _vec(out, "out", n), n,
                                 _stream(stream)), "gguf_swiglu_f32")
    return out


def gguf_add_f32(a, b, out=None, stream=None):
    """out = a + b."""
    n = a.numel()
    out = torch.empty_like(a) if out is None else out
    _check(lib().gguf_add_f32(_vec(a, "a"), _vec(b, "b", n), _vec(out, "out", n), n, _stream(stream)),
           "gguf_add_f32")
    return out


# ------------------------------------------------- paged key-value cache (include/gguf_kv.h)

_F32 = (torch.float32,)
_SOURCES = (torch.float32, torch.bfloat16)


class KvCacheStruct(ctypes.Structure):
    """struct gguf_kv_cache of the C ABI."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("pos", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("type", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class KvCache:
    """One layer's paged key-value cache: device tensors the caller owns (`k` and
    `v` of n_pages * gguf_kv_page_bytes(...) bytes each, any dtype; optional
    `weight` fp32 and `pos` int32 planes of n_pages * n_kv_heads * page_size) and
    the C description of them. The layout is in include/gguf_kv.h. Keeps the
    tensors alive.

    type is TENSOR_F16, TENSOR_BF16 or TYPE_Q8_0. KvCache.empty allocates."""

    def __init__(self, k, v, type, n_kv_heads, head_dim, page_size, weight=None, pos=None):
        page = gguf_kv_page_bytes(type, n_kv_heads, head_dim, page_size)
        if page < 0:
            raise GgufQkArgumentError(page, "KvCache")
        kp, vp = _dev(k, "k"), _dev(v, "v")
        self.device = k.get_device()   # index
        nbytes = k.numel() * k.element_size()
        if nbytes == 0 or nbytes % page:
            raise ValueError(f"k holds {nbytes} bytes, not whole pages of {page}")
        if v.numel() * v.element_size() != nbytes:
            raise ValueError("k and v must hold the same number of bytes")
        self.n_pages = nbytes // page
        slots = self.n_pages * n_kv_heads * page_size
        for t, name, dt in ((weight, "weight", torch.float32), (pos, "pos", torch.int32)):
            if t is not None:
                _tensor(t, name, self.device, dt)
                if t.numel() != slots:
                    raise ValueError(f"{name} holds {t.numel()} values, expected {slots}")
        if v.get_device() != self.device:
            raise ValueError("k and v must be on one device")
        self.k, self.v, self.weight, self.pos = k, v, weight, pos
        self.type, self.n_kv_heads, self.head_dim, self.page_size = type, n_kv_heads, head_dim, page_size
        self.struct = KvCacheStruct(kp, vp, None if weight is None else weight.data_ptr(),
                                    None if pos is None else pos.data_ptr(), self.n_pages, type, n_kv_heads,
                                    head_dim, page_size)
        self.address = ctypes.addressof(self.struct)

    @classmethod
    def empty(cls, type, n_pages, n_kv_heads, head_dim, page_size, device="cuda:0", planes=False):
        """A cache of zeros; with `planes` it has weight and pos (for eviction)."""
        page = gguf_kv_page_bytes(type, n_kv_heads, head_dim, page_size)
        if page < 0:
            raise GgufQkArgumentError(page, "KvCache.empty")
        k, v = (torch.zeros(n_pages * page, dtype=torch.uint8, device=device) for _ in range(2))
        w = p = None
        if planes:
            w = torch.zeros((n_pages, n_kv_heads, page_size), dtype=torch.float32, device=device)
            p = torch.zeros((n_pages, n_kv_heads, page_size), dtype=torch.int32, device=device)
        return cls(k, v, type, n_kv_heads, head_dim, page_size, weight=w, pos=p)


def _tensor(t, name, device, dtype=None):
    """The address of a contiguous tensor on device `device` (index). These calls
    run once per decode step: the checks stay few and cheap."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be a tensor on device {device}, got {t.device}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, device, row, dtypes):
    """(address, row stride) of [n, row] or [n, heads, dim] values whose rows may lie apart."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be a tensor on device {device}, got {t.device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {dtypes}, got {t.dtype}")
    shape = t.shape
    if len(shape) not in (2, 3) or math.prod(shape[1:]) != row:
        raise ValueError(f"{name} must be rows of {row} values, got {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), row
    stride = t.stride()
    if (row > 1 and stride[-1] != 1 and shape[-1] > 1) or (
            len(shape) == 3 and shape[1] > 1 and stride[1] != shape[2]):
        raise ValueError(f"{name} must be rows of {row} consecutive values, got strides {stride}")
    return t.data_ptr(), (stride[0] if shape[0] > 1 else row)


def _ints(t, name, device, n):
    p = _tensor(t, name, device, torch.int32)
    if t.numel() != n:
        raise ValueError(f"{name} holds {t.numel()} values, expected {n}")
    return p


def _table(t, device):
    p = _tensor(t, "page_table", device, torch.int32)
    if t.dim() != 2 or t.shape[1] < 1:
        raise ValueError("page_table must be [n_seqs, pages]")
    return p


def _call(device, stream, run):
    """Runs run(stream handle) with the tensors' device (index) current (the library
    works on the current device) and, where a stream is given, that stream current
    for what run allocates."""
    if stream is None and torch._C._cuda_getDevice() == device:
        return run(torch._C._cuda_getCurrentRawStream(device))
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != device:
        raise ValueError(f"stream is on device {stream.device_index}, the tensors are on device {device}")
    with contextlib.ExitStack() as on:
        on.enter_context(torch.cuda.device(device))
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)
            on.enter_context(torch.cuda.stream(stream))
        return run(torch._C._cuda_getCurrentRawStream(device))


def _work(workspace, need, device):
    """(tensor, address, bytes) of a workspace: the caller's, or one of the call's
    own, of the bytes need() says."""
    if workspace is None:
        n = need()
        if n < 0:
            raise GgufQkArgumentError(n, "workspace")
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=torch.device("cuda", device))
    return workspace, _tensor(workspace, "workspace", device), workspace.numel() * workspace.element_size()


def gguf_kv_page_bytes(type_id: int, n_kv_heads: int, head_dim: int, page_size: int) -> int:
    """Bytes of one page of K (and of V), or a negative status."""
    return lib().gguf_kv_page_bytes(type_id, n_kv_heads, head_dim, page_size)


def gguf_kv_append(cache: KvCache, k, v, page_table, slot, seq=None, pos=None, stream=None):
    """Write tokens (rows of k and v, fp32 or bf16 [n_tokens, n_kv_heads * head_dim],
    rows may lie apart) to slot[t] of sequence seq[t] (None: t). A token with a
    slot or seq out of range is dropped. pos: the tokens' positions where the cache
    keeps them (None: the slots, right only before a sequence's first eviction)."""
    row, dev = cache.n_kv_heads * cache.head_dim, cache.device
    (kp, ks), (vp, vs) = _rows(k, "k", dev, row, _SOURCES), _rows(v, "v", dev, row, _SOURCES)
    n = k.shape[0]
    if v.shape[0] != n or v.dtype is not k.dtype or ks != vs:
        raise ValueError("k and v must have the same rows, type and row stride")
    tp, sp = _table(page_table, dev), _ints(slot, "slot", dev, n)
    qp = None if seq is None else _ints(seq, "seq", dev, n)
    pp = None if pos is None else _ints(pos, "pos", dev, n)
    src = TENSOR_F32 if k.dtype is torch.float32 else TENSOR_BF16
    if n == 0:   # empty tensors have no address
        return
    seqs, pages = page_table.shape
    _check(_call(dev, stream, lambda st: lib().gguf_kv_append(
        cache.address, kp, vp, src, ks, n, qp, sp, pp, tp, pages, seqs, st)), "gguf_kv_append")


def gguf_attn_decode_workspace(cache: KvCache, n_seqs: int, n_heads: int, max_len: int, track: bool = False) -> int:
    """Bytes of workspace of gguf_attn_decode calls with at most n_seqs sequences, at
    most max_len and any window, or a negative status."""
    return lib().gguf_attn_decode_workspace(cache.address, n_seqs, n_heads, max_len, int(track))


def gguf_attn_decode(cache: KvCache, q, page_table, lengths, max_len, scale=None, window=0, track=False, out=None,
                     workspace=None, stream=None):
    """Attention of one new token per sequence: q fp32 [n_seqs, n_heads, head_dim] or
    [n_seqs, n_heads * head_dim] over the first lengths[s] slots of the cache
    (the last `window` of them where given: slots, which are the newest tokens only
    until an eviction reorders them; gguf_kv_evict with budget = recent = the window
    keeps a window of positions), scale 1 / sqrt(head_dim) unless given. Returns
    out, fp32 of q's shape. With `track` the cache's weight grows
    by the attention each slot received. `workspace`: a tensor of at least
    gguf_attn_decode_workspace bytes that no overlapping call uses (None: the
    call allocates one)."""
    d, dev, shape = cache.head_dim, cache.device, q.shape
    n, row = shape[0], math.prod(shape[1:])
    if row == 0 or row % d:
        raise ValueError("q must be [n_seqs, n_heads, head_dim]")
    heads = row // d
    qp, qs = _rows(q, "q", dev, row, _F32)
    tp, lp = _table(page_table, dev), _ints(lengths, "lengths", dev, n)
    seqs, pages = page_table.shape
    if seqs != n:
        raise ValueError("one row of page_table per sequence")
    scale = d ** -0.5 if scale is None else scale

    def run(st):
        o = torch.empty(shape, dtype=torch.float32, device=q.device) if out is None else out
        op, os_ = _rows(o, "out", dev, row, _F32)
        if o.shape[0] != n:
            raise ValueError("out must have one row per sequence")
        if n == 0:   # empty tensors have no address
            return o
        ws, wp, wn = _work(workspace, lambda: gguf_attn_decode_workspace(cache, n, heads, max_len, track), dev)
        _check(lib().gguf_attn_decode(cache.address, qp, qs, op, os_, n, heads, tp, pages, lp, max_len, scale, window,
                                      1 if track else 0, wp, wn, st), "gguf_attn_decode")
        return o
    return _call(dev, stream, run)


def gguf_kv_evict_workspace(cache: KvCache, n_seqs: int, max_len: int, budget: int) -> int:
    """Bytes of workspace of a gguf_kv_evict call, or a negative status."""
    return lib().gguf_kv_evict_workspace(cache.address, n_seqs, max_len, budget)


def gguf_kv_evict(cache: KvCache, page_table, lengths, max_len, budget, recent=0, workspace=None, stream=None):
    """Cut every sequence longer than `budget` to the `budget` slots per kv head
    that received most attention (the newest `recent` tokens always stay). Moves
    the kept slots behind the budget into the vacated ones and updates lengths; the
    slots are then no longer in the order of positions. max_len has to bound every
    length: what lies behind it in a longer sequence is lost, `recent` tokens too."""
    dev = cache.device
    tp = _table(page_table, dev)
    n, pages = page_table.shape
    lp = _ints(lengths, "lengths", dev, n)
    if n == 0:
        return

    def run(st):
        ws, wp, wn = _work(workspace, lambda: gguf_kv_evict_workspace(cache, n, max_len, budget), dev)
        _check(lib().gguf_kv_evict(cache.address, n, tp, pages, lp, max_len, budget, recent, wp, wn, st),
               "gguf_kv_evict")
    _call(dev, stream, run)


class Logprobs(NamedTuple):
    """What gguf_logprobs returns (None for a part that was not asked for)."""
    token_logprobs: Optional[torch.Tensor]   # fp32 [n_rows, n_tokens]
    entropy: torch.Tensor                    # fp32 [n_rows]
    top_ids: Optional[torch.Tensor]          # int32 [n_rows, top_k]
    top_logprobs: Optional[torch.Tensor]     # fp32 [n_rows, top_k]


def gguf_logprobs_workspace(n_rows: int, vocab: int, top_k: int) -> int:
    """Bytes of workspace of a gguf_logprobs call, or a negative status."""
    return lib().gguf_logprobs_workspace(n_rows, vocab, top_k)


def gguf_logprobs(logits, tokens=None, top_k=0, workspace=None, stream=None) -> Logprobs:
    """Log probabilities of the given tokens (int32 [n_rows, n_tokens], or flat: one
    per row, or those of the one row) under logits (fp32 or bf16 [n_rows, vocab] or [vocab], rows may lie apart),
    the entropy of each row, and its top_k tokens with theirs."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch tensor")
    x = logits.unsqueeze(0) if logits.dim() == 1 else logits
    if x.dim() != 2:
        raise ValueError("logits must be [n_rows, vocab]")
    if not x.is_cuda:
        raise ValueError("logits must be a device tensor")
    dev = x.get_device()
    n, vocab = x.shape
    xp, xs = _rows(x, "logits", dev, vocab, _SOURCES)
    m, tp = 0, None
    if tokens is not None:
        tp = _tensor(tokens, "tokens", dev, torch.int32)
        # a flat list: one token per row, or the tokens of the one row
        shape = tuple(tokens.shape) if tokens.dim() != 1 else (1, len(tokens)) if n == 1 else (len(tokens), 1)
        if len(shape) != 2 or shape[0] != n:
            raise ValueError("tokens must be [n_rows, n_tokens] or [n_rows]")
        m = shape[1]

    def run(st):
        new = x.new_empty
        ent = new((n,), dtype=torch.float32)
        lp = new((n, m), dtype=torch.float32) if m else None
        ids = new((n, top_k), dtype=torch.int32) if top_k else None
        top = new((n, top_k), dtype=torch.float32) if top_k else None
        if n:
            ws, wp, wn = _work(workspace, lambda: gguf_logprobs_workspace(n, vocab, top_k), dev)
            _check(lib().gguf_logprobs(xp, TENSOR_F32 if x.dtype is torch.float32 else TENSOR_BF16, n, vocab, xs, tp,
                                       m, top_k, lp.data_ptr() if m else None, ent.data_ptr(),
                                       ids.data_ptr() if top_k else None, top.data_ptr() if top_k else None, wp, wn,
                                       st), "gguf_logprobs")
        return Logprobs(lp, ent, ids, top)
    if not 0 <= top_k <= vocab:
        raise GgufQkArgumentError(ERR_SHAPE, "top_k")
    return _call(dev, stream, run)


class RopeStruct(ctypes.Structure):
    """struct gguf_rope of the C ABI."""
    _fields_ = [("freqs", ctypes.c_void_p), ("axes", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("pos_stride", ctypes.c_int64), ("n_axes", ctypes.c_int32), ("n_rot", ctypes.c_int32),
                ("pairing", ctypes.c_int32), ("magnitude", ctypes.c_float)]


ROPE_ADJACENT, ROPE_HALVES = 0, 1


def gguf_qk_rope(q, k, pos=None, freqs=None, axes=None, halves=True, magnitude=1.0, q_norm=None, k_norm=None, eps=1e-6,
                 q_out=None, k_out=None, stream=None):
    """Norms of queries and keys per head (weights q_norm, k_norm: fp32 [head_dim]) and
    the rotation by position. q [n_tokens, n_heads, head_dim] and k [n_tokens,
    n_kv_heads, head_dim] (either may be None), fp32 or bf16, rows may lie apart. pos
    int32 [n_tokens], or [n_axes, n_tokens] with axes int32 [len(freqs)] naming each
    pair's axis; freqs fp64 [n_rot / 2] radians per position (both None: norms only).
    halves: pair i is elements i and i + n_rot / 2, else 2 i and 2 i + 1. Returns
    (q_out, k_out), which may be given (q and k themselves: in place)."""
    one = k if q is None else q
    if one is None:
        raise ValueError("q or k must be given")
    for x in (q, k):
        if x is not None and not isinstance(x, torch.Tensor):
            raise TypeError("q and k must be torch tensors")
    if one.dim() != 3:
        raise ValueError("q and k must be [n_tokens, n_heads, head_dim]")
    dev, dt = one.get_device(), one.dtype
    n, _, d = one.shape
    if dev < 0:
        raise ValueError("q and k must be device tensors")
    type_id = _source_id(dt)
    if (pos is None) != (freqs is None) or (axes is not None and freqs is None):
        raise ValueError("pos and freqs belong together, and axes to them")
    ref = None
    if freqs is not None:
        fp, half = _tensor(freqs, "freqs", dev, torch.float64), freqs.numel()
        pp, shape = _tensor(pos, "pos", dev, torch.int32), pos.shape
        if len(shape) not in (1, 2) or shape[-1] != n:
            raise ValueError("pos must be [n_tokens] or [n_axes, n_tokens]")
        ap = None if axes is None else _ints(axes, "axes", dev, half)
        rope = RopeStruct(fp, ap, pp, n, 1 if len(shape) == 1 else shape[0], 2 * half,
                          ROPE_HALVES if halves else ROPE_ADJACENT, magnitude)
        ref = ctypes.addressof(rope)
    qw = None if q_norm is None else _floats(q_norm, "q_norm", dev, d)
    kw = None if k_norm is None else _floats(k_norm, "k_norm", dev, d)

    def rows(x, name):
        """(address, row stride, heads)"""
        shape = x.shape
        if len(shape) != 3 or shape[0] != n or shape[2] != d or x.dtype is not dt:
            raise ValueError("q and k must be of one type, with the same tokens and head_dim")
        return *_rows(x, name, dev, shape[1] * d, (dt,)), shape[1]

    def run(st):
        qo, ko, qp, kp, qop, kop, qs, ks, qos, kos, qh, kh = q_out, k_out, None, None, None, None, 0, 0, 0, 0, 0, 0
        if q is not None:
            qp, qs, qh = rows(q, "q")
            if qo is None:
                qo = torch.empty(q.shape, dtype=dt, device=q.device)
            qop, qos, h = rows(qo, "q_out")
            if h != qh:
                raise ValueError("q_out must have q's shape")
        if k is not None:
            kp, ks, kh = rows(k, "k")
            if ko is None:
                ko = torch.empty(k.shape, dtype=dt, device=k.device)
            kop, kos, h = rows(ko, "k_out")
            if h != kh:
                raise ValueError("k_out must have k's shape")
        if n:   # empty tensors have no address
            _check(lib().gguf_qk_rope(qp, qs, qop, qos, qh, kp, ks, kop, kos, kh, type_id, n, d, qw, kw, eps, ref, st),
                   "gguf_qk_rope")
        return None if q is None else qo, None if k is None else ko
    return _call(dev, stream, run)


def _source_id(dtype):
    if dtype not in _SOURCES:
        raise ValueError(f"expected fp32 or bf16, got {dtype}")
    return TENSOR_F32 if dtype is torch.float32 else TENSOR_BF16


def gguf_attn_extend_workspace(cache: KvCache, dtype, n_seqs: int, n_rows: int, n_heads: int, max_len: int,
                               window: int = 0, sinks: int = 0) -> int:
    """Bytes of workspace of gguf_attn_extend calls with queries of this dtype, at most
    n_seqs sequences, n_rows rows and max_len, and this window and sinks, or a negative
    status."""
    return lib().gguf_attn_extend_workspace(cache.address, _source_id(dtype), n_seqs, n_rows, n_heads, max_len, window,
                                            sinks)


def gguf_attn_extend(cache: KvCache, q, page_table, lengths, max_len, row_start=None, scale=None, window=0, sinks=0,
                     out=None, workspace=None, stream=None):
    """Attention of the newest tokens of each sequence over the cache that holds them:
    q fp32 or bf16 [n_rows, n_heads, head_dim] or [n_rows, n_heads * head_dim], the rows
    of sequence s from row_start[s] to row_start[s + 1] - 1 (int32 [n_seqs + 1]; None:
    one row per sequence), the last of them at slot lengths[s] - 1. A row sees the slots
    up to its own; with a window the last `window` of those and the first `sinks` of the
    sequence. scale 1 / sqrt(head_dim) unless given. Returns out, of q's shape and type
    (rows of no sequence are left as they were). A long sequence with few rows is better
    passed apart from prompts: the call's totals choose its one kernel and its splits. `workspace`: a tensor of at least
    gguf_attn_extend_workspace bytes that no overlapping call uses (None: the call
    allocates one)."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch tensor")
    d, dev, shape = cache.head_dim, cache.device, q.shape
    rows, row = shape[0], math.prod(shape[1:])
    if row == 0 or row % d:
        raise ValueError("q must be [n_rows, n_heads, head_dim]")
    heads, type_id = row // d, _source_id(q.dtype)
    qp, qs = _rows(q, "q", dev, row, (q.dtype,))
    tp = _table(page_table, dev)
    seqs, pages = page_table.shape
    lp = _ints(lengths, "lengths", dev, seqs)
    rp = None if row_start is None else _ints(row_start, "row_start", dev, seqs + 1)
    if row_start is None and rows != seqs:
        raise ValueError("one row per sequence unless row_start is given")
    scale = d ** -0.5 if scale is None else scale

    def run(st):
        o = torch.empty(shape, dtype=q.dtype, device=q.device) if out is None else out
        op, os_ = _rows(o, "out", dev, row, (q.dtype,))
        if o.shape[0] != rows:
            raise ValueError("out must have q's rows")
        if rows == 0 or seqs == 0:   # empty tensors have no address
            return o
        ws, wp, wn = _work(workspace, lambda: gguf_attn_extend_workspace(cache, q.dtype, seqs, rows, heads, max_len,
                                                                         window, sinks), dev)
        _check(lib().gguf_attn_extend(cache.address, qp, type_id, qs, op, os_, rp, rows, seqs, heads, tp, pages, lp,
                                      max_len, scale, window, sinks, wp, wn, st), "gguf_attn_extend")
        return o
    return _call(dev, stream, run)


class Verified(NamedTuple):
    """What gguf_verify_draft returns."""
    accepted: torch.Tensor      # int32 [n_seqs]: drafted tokens accepted
    next_tokens: torch.Tensor   # int32 [n_seqs]: the token behind them
    accept_prob: torch.Tensor   # fp32 [n_rows]: each drafted token's probability of acceptance


def gguf_verify_draft_workspace(n_rows: int, n_seqs: int, vocab: int, has_draft: bool) -> int:
    """Bytes of workspace of a gguf_verify_draft call, or a negative status."""
    return lib().gguf_verify_draft_workspace(n_rows, n_seqs, vocab, int(has_draft))


def gguf_verify_draft(target, tokens, uniform, uniform_next, row_start, draft=None, temperature=None, workspace=None,
                      stream=None) -> Verified:
    """Which drafted tokens the target accepts, and the token behind them, from given
    random numbers. target and draft: logits, fp32 or bf16 [n_rows, vocab], rows may lie
    apart (draft None: drafts without probabilities); the rows of sequence s are
    row_start[s] to row_start[s + 1] - 1 (int32 [n_seqs + 1]), one per drafted token and
    a last one. tokens int32 and uniform fp32 [n_rows] (the last rows' are not looked
    at), uniform_next fp32 [n_seqs], temperature fp32 [n_seqs] (0: greedy; None: 1)."""
    if not isinstance(target, torch.Tensor):
        raise TypeError("target must be a torch tensor")
    if target.dim() != 2 or not target.is_cuda:
        raise ValueError("target must be a device tensor [n_rows, vocab]")
    dev, (n, vocab), type_id = target.get_device(), target.shape, _source_id(target.dtype)
    xp, xs = _rows(target, "target", dev, vocab, (target.dtype,))
    yp, ys = None, 0
    if draft is not None:
        yp, ys = _rows(draft, "draft", dev, vocab, (target.dtype,))
        if draft.shape != target.shape:
            raise ValueError("draft must have target's shape")
    sp = _tensor(row_start, "row_start", dev, torch.int32)
    seqs = row_start.numel() - 1
    if seqs < 0:
        raise ValueError("row_start must hold n_seqs + 1 values")
    tp, up = _ints(tokens, "tokens", dev, n), _floats(uniform, "uniform", dev, n)
    np_ = _floats(uniform_next, "uniform_next", dev, seqs)
    cp = None if temperature is None else _floats(temperature, "temperature", dev, seqs)

    def run(st):
        new = target.new_empty
        accepted, nxt = new((seqs,), dtype=torch.int32), new((seqs,), dtype=torch.int32)
        prob = new((n,), dtype=torch.float32)
        if seqs:
            ws, wp, wn = _work(workspace, lambda: gguf_verify_draft_workspace(n, seqs, vocab, draft is not None), dev)
            _check(lib().gguf_verify_draft(xp, xs, yp, ys, type_id, tp, up, np_, sp, n, seqs, vocab, cp,
                                           accepted.data_ptr(), nxt.data_ptr(), prob.data_ptr() if n else None, wp, wn,
                                           st), "gguf_verify_draft")
        return Verified(accepted, nxt, prob)
    return _call(dev, stream, run)


def _floats(t, name, device, n):
    p = _tensor(t, name, device, torch.float32)
    if t.numel() != n:
        raise ValueError(f"{name} holds {t.numel()} values, expected {n}")
    return p


# ------------------------------------------------------------------ GGUF files

def gguf_tensor_nbytes(type_id: int, dims) -> int:
    """Bytes of a tensor of this type and dims (fastest first), or a negative status."""
    d = (ctypes.c_int64 * 4)(*([int(v) for v in dims] + [1] * (4 - len(dims))))
    return lib().gguf_tensor_nbytes(type_id, len(dims), d)


def gguf_file_open(path):
    """Maps and parses a GGUF file; returns the library handle (ctypes.c_void_p)."""
    h = ctypes.c_void_p()
    _check(lib().gguf_file_open(os.fsencode(os.fspath(path)), ctypes.byref(h)), "gguf_file_open")
    return h


def gguf_file_close(h) -> None:
    lib().gguf_file_close(h)


def gguf_file_version(h) -> int:
    return lib().gguf_file_version(h)


def gguf_file_tensor_count(h) -> int:
    return lib().gguf_file_tensor_count(h)


def gguf_file_kv_count(h) -> int:
    return lib().gguf_file_kv_count(h)


def gguf_file_alignment(h) -> int:
    return lib().gguf_file_alignment(h)


def gguf_file_data_offset(h) -> int:
    return lib().gguf_file_data_offset(h)


def gguf_file_size(h) -> int:
    return lib().gguf_file_size(h)


def gguf_file_tensor(h, i: int) -> GgufTensorInfo:
    info = GgufTensorInfo()
    _check(lib().gguf_file_tensor(h, i, ctypes.byref(info)), "gguf_file_tensor")
    return info


def gguf_file_kv(h, i: int) -> GgufKvInfo:
    info = GgufKvInfo()
    _check(lib().gguf_file_kv(h, i, ctypes.byref(info)), "gguf_file_kv")
    return info


def gguf_file_find_tensor(h, name: str) -> int:
    """Index of the tensor, or ERR_NOT_FOUND."""
    return lib().gguf_file_find_tensor(h, name.encode())


def gguf_file_find_kv(h, key: str) -> int:
    """Index of the metadata entry, or ERR_NOT_FOUND."""
    return lib().gguf_file_find_kv(h, key.encode())


def gguf_file_kv_array_string(h, i: int, j: int) -> bytes:
    p, n = ctypes.c_void_p(), ctypes.c_int64()
    _check(lib().gguf_file_kv_array_string(h, i, j, ctypes.byref(p), ctypes.byref(n)),
           "gguf_file_kv_array_string")
    return ctypes.string_at(p, n.value) if n.value else b""


def gguf_file_upload_tensor(h, i: int, dst: torch.Tensor, stream=None) -> torch.Tensor:
    """Copies tensor i's raw bytes into the uint8 device tensor dst."""
    _check(lib().gguf_file_upload_tensor(h, i, _dev(dst, "dst", torch.uint8), _stream(stream)),
           "gguf_file_upload_tensor")
    return dst


class GgufFile:
    """A GGUF file mapped and parsed by the library (include/gguf_file.h).

    `tensors` lists the tensor records (name, type, dims fastest first, absolute
    offset, nbytes); `metadata` decodes every entry (scalars, strings, arrays of
    scalars or strings; nested arrays are returned as their raw payload bytes);
    `upload` copies a tensor's raw bytes to a new device tensor through the
    library. Use as a context manager or call close()."""

    def __init__(self, path):
        self._h = gguf_file_open(path)

    def close(self):
        if getattr(self, "_h", None):
            gguf_file_close(self._h)
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        self.close()

    def _handle(self):
        if not self._h:
            raise ValueError("the file is closed")
        return self._h

    @property
    def version(self) -> int:
        return gguf_file_version(self._handle())

    @property
    def alignment(self) -> int:
        return gguf_file_alignment(self._handle())

    @property
    def data_offset(self) -> int:
        return gguf_file_data_offset(self._handle())

    @property
    def size(self) -> int:
        return gguf_file_size(self._handle())

    def _index(self, name_or_index) -> int:
        if isinstance(name_or_index, int):
            return name_or_index
        i = gguf_file_find_tensor(self._handle(), name_or_index)
        if i < 0:
            raise KeyError(name_or_index)
        return i

    def tensor(self, name_or_index) -> dict:
        info = gguf_file_tensor(self._handle(), self._index(name_or_index))
        return {"name": info.name.decode("utf-8", "replace"), "type": info.type,
                "dims": tuple(info.dims[: info.n_dims]), "offset": info.offset,
                "nbytes": info.nbytes, "host_ptr": info.data}

    @property
    def tensors(self) -> list:
        return [self.tensor(i) for i in range(gguf_file_tensor_count(self._handle()))]

    def _kv_value(self, i: int, info: GgufKvInfo):
        raw = ctypes.string_at(info.data, info.nbytes) if info.nbytes else b""
        if info.type in _SCALAR_FMT:
            return struct.unpack(_SCALAR_FMT[info.type], raw)[0]
        if info.type == VALUE_STRING:
            return raw.decode("utf-8", "replace")
        if info.type == VALUE_ARRAY:
            if info.elem_type in _SCALAR_FMT:
                fmt = _SCALAR_FMT[info.elem_type]
                return list(struct.unpack("<%d%s" % (info.count, fmt[1]), raw))
            if info.elem_type == VALUE_STRING:
                return [gguf_file_kv_array_string(self._handle(), i, j).decode("utf-8", "replace")
                        for j in range(info.count)]
            return raw
        raise GgufQkArgumentError(ERR_FORMAT, "metadata value")

    @property
    def metadata(self) -> dict:
        out = {}
        for i in range(gguf_file_kv_count(self._handle())):
            info = gguf_file_kv(self._handle(), i)
            out[info.key.decode("utf-8", "replace")] = self._kv_value(i, info)
        return out

    def kv_type(self, key: str):
        """(value type, element type) of a metadata entry."""
        i = gguf_file_find_kv(self._handle(), key)
        if i < 0:
            raise KeyError(key)
        info = gguf_file_kv(self._handle(), i)
        return info.type, info.elem_type

    def upload(self, name_or_index, device="cuda:0", stream=None):
        """A new uint8 device tensor [nbytes] holding the tensor's raw bytes."""
        i = self._index(name_or_index)
        t = self.tensor(i)
        if t["nbytes"] < 0:
            raise GgufQkArgumentError(ERR_FORMAT, f"tensor {t['name']} has a type of unknown size")
        out = torch.empty(max(t["nbytes"], 16), dtype=torch.uint8, device=device)
        gguf_file_upload_tensor(self._handle(), i, out, stream)
        return out[: t["nbytes"]]
