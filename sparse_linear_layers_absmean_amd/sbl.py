"""Thin Python binding of libsbl (include/sbl.h) over PyTorch device tensors.

Argument marshalling only: every step of the path runs in the HIP kernels of
libsbl.so.  PyTorch supplies device memory and the current HIP stream.  The
binding checks that each tensor is on the GPU, contiguous, of the right dtype
and large enough for the sizes passed, so a kernel can never be handed a
buffer smaller than it will touch.  There is no CPU fallback: if the library
is missing, loading fails loudly.
"""

from __future__ import annotations

import ctypes
import os

import torch  # loaded first so libsbl binds to the same HIP runtime

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsbl.so")

SBL_OK = 0
SBL_FMT_DENSE2 = 0
SBL_FMT_NM = 1
# weight-preparation variants and execution choices (sbl_quant_weights_batch_ex flags)
SBL_QW_DEFAULT, SBL_QW_BETA_KEPT, SBL_QW_MASK_FROM_CODES = 0, 1, 2
SBL_QW_TWO_PASS, SBL_QW_NO_WAIT = 4, 8
# numeric types of dense operands (sbl_dtype); the output head's losses take the 16-bit ones
SBL_BF16, SBL_FP16, SBL_FP32 = 0, 1, 2
ABI_VERSION = 11

_c_i64 = ctypes.c_int64
_c_i32 = ctypes.c_int32
_c_p = ctypes.c_void_p

_lib = None


class LinearItem(ctypes.Structure):
    """sbl_linear_item of include/sbl.h."""
    _fields_ = [("packed", _c_p), ("meta", _c_p), ("beta", _c_p), ("xq", _c_p), ("gamma", _c_p),
                ("m_tok", _c_i64), ("n_out", _c_i64), ("k", _c_i64), ("y", _c_p), ("acc", _c_p)]


class QuantItem(ctypes.Structure):
    """sbl_quant_item of include/sbl.h."""
    _fields_ = [("w_bf16", _c_p), ("n_out", _c_i64), ("k", _c_i64), ("beta", _c_p),
                ("mask_bits", _c_p), ("codes", _c_p), ("packed", _c_p), ("meta", _c_p),
                ("workspace", _c_p), ("workspace_bytes", _c_i64)]


class AdamWItem(ctypes.Structure):
    """sbl_adamw_item of include/sbl.h."""
    _fields_ = [("w", _c_p), ("w_low", _c_p), ("g", _c_p), ("m", _c_p), ("v", _c_p), ("m_scale", _c_p), ("v_scale", _c_p),
                ("n", _c_i64), ("w_dtype", _c_i32), ("g_dtype", _c_i32), ("state_bits", _c_i32),
                ("lr_scale", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class SblError(RuntimeError):
    def __init__(self, func: str, status: int):
        lib = load()
        msg = lib.sbl_status_string(status).decode()
        if status == 5:
            msg += f" (hip error {lib.sbl_last_hip_error()})"
        super().__init__(f"{func}: status {status}: {msg}")
        self.status = status


def load():
    """Load libsbl.so (built in-tree by build.py / __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    try:
        lib.sbl_abi_version.restype = ctypes.c_int
        if lib.sbl_abi_version() != ABI_VERSION:
            raise RuntimeError("libsbl.so ABI version mismatch: rebuild it")
        _declare(lib)
    except AttributeError as e:                      # built before the newest functions
        raise RuntimeError(f"libsbl.so is older than its binding ({e}): rebuild it") from e
    _lib = lib
    return lib


def _declare(lib):
    """Argument and result types of every function."""
    lib.sbl_status_string.restype = ctypes.c_char_p
    lib.sbl_status_string.argtypes = [ctypes.c_int]
    lib.sbl_last_hip_error.restype = ctypes.c_int
    lib.sbl_packed_bytes.restype = _c_i64
    lib.sbl_packed_bytes.argtypes = [_c_i64, _c_i64, _c_i32, _c_i32, _c_i32]
    lib.sbl_meta_bytes.restype = _c_i64
    lib.sbl_meta_bytes.argtypes = [_c_i64, _c_i64, _c_i32]
    lib.sbl_workspace_bytes.restype = _c_i64
    lib.sbl_workspace_bytes.argtypes = [_c_i64, _c_i64]
    lib.sbl_workspace_init.restype = ctypes.c_int
    lib.sbl_workspace_init.argtypes = [_c_p, _c_i64, _c_p]
    lib.sbl_quant_weights.restype = ctypes.c_int
    lib.sbl_quant_weights.argtypes = [_c_p, _c_i64, _c_i64, _c_i32, _c_i32, _c_p, _c_p, _c_p,
                                      _c_i32, _c_p, _c_p, _c_p, _c_i64, _c_p]
    lib.sbl_quant_weights_batch.restype = ctypes.c_int
    lib.sbl_quant_weights_batch.argtypes = [ctypes.POINTER(QuantItem), _c_i32, _c_i32, _c_i32, _c_i32,
                                            _c_p]
    lib.sbl_quant_weights_batch_ex.restype = ctypes.c_int
    lib.sbl_quant_weights_batch_ex.argtypes = [ctypes.POINTER(QuantItem), _c_i32, _c_i32, _c_i32, _c_i32,
                                               _c_i32, _c_p]
    lib.sbl_quant_weights_batch_noalloc.restype = ctypes.c_int
    lib.sbl_quant_weights_batch_noalloc.argtypes = [ctypes.POINTER(QuantItem), _c_i32, _c_i32, _c_i32, _c_i32,
                                                    _c_p]
    lib.sbl_pack.restype = ctypes.c_int
    lib.sbl_pack.argtypes = [_c_p, _c_p, _c_i64, _c_i64, _c_i32, _c_i32, _c_i32, _c_p, _c_p, _c_p]
    lib.sbl_quant_acts.restype = ctypes.c_int
    lib.sbl_quant_acts.argtypes = [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p]
    lib.sbl_linear.restype = ctypes.c_int
    lib.sbl_linear.argtypes = [_c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_p, _c_p, _c_p,
                               _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p]
    lib.sbl_linear_batch.restype = ctypes.c_int
    lib.sbl_linear_batch.argtypes = [ctypes.POINTER(LinearItem), _c_i32, _c_i32, _c_i32, _c_i32, _c_p]
    lib.sbl_linear_acts_batch.restype = ctypes.c_int
    lib.sbl_linear_acts_batch.argtypes = [_c_p, _c_i64, _c_i64, _c_p, _c_p, ctypes.POINTER(LinearItem),
                                          _c_i32, _c_i32, _c_i32, _c_i32, _c_p]
    lib.sbl_workspace_bytes_grouped.restype = _c_i64
    lib.sbl_workspace_bytes_grouped.argtypes = [_c_i64, _c_i64, _c_i64]
    lib.sbl_quant_weights_grouped.restype = ctypes.c_int
    lib.sbl_quant_weights_grouped.argtypes = [_c_p, _c_i64, _c_i64, _c_i32, _c_i32, _c_i64, _c_p, _c_p, _c_p,
                                              _c_i32, _c_p, _c_p, _c_p, _c_i64, _c_p]
    lib.sbl_linear_grouped.restype = ctypes.c_int
    lib.sbl_linear_grouped.argtypes = [_c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_p, _c_i64, _c_p, _c_p,
                                       _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p]
    lib.sbl_quant_acts_kgrouped.restype = ctypes.c_int
    lib.sbl_quant_acts_kgrouped.argtypes = [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p]
    lib.sbl_workspace_bytes_blocked.restype = _c_i64
    lib.sbl_workspace_bytes_blocked.argtypes = [_c_i64, _c_i64, _c_i64, _c_i64]
    lib.sbl_quant_weights_blocked.restype = ctypes.c_int
    lib.sbl_quant_weights_blocked.argtypes = [_c_p, _c_i64, _c_i64, _c_i32, _c_i32, _c_i64, _c_i64, _c_p, _c_p, _c_p,
                                              _c_i32, _c_p, _c_p, _c_p, _c_i64, _c_p]
    lib.sbl_linear_blocked.restype = ctypes.c_int
    lib.sbl_linear_blocked.argtypes = [_c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_p, _c_i64, _c_p, _c_p, _c_i64,
                                       _c_i64, _c_i64, _c_i64, _c_p, _c_p]
    lib.sbl_linear_kgrouped.restype = ctypes.c_int
    lib.sbl_linear_kgrouped.argtypes = [_c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_p, _c_i64, _c_p, _c_p, _c_i64,
                                        _c_i64, _c_i64, _c_i64, _c_p, _c_p]
    lib.sbl_linear_backward.restype = ctypes.c_int
    lib.sbl_linear_backward.argtypes = [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i32, _c_i32, _c_i32,
                                        _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]
    lib.sbl_backward_workspace_bytes.restype = ctypes.c_int64
    lib.sbl_backward_workspace_bytes.argtypes = [_c_i64, _c_i64, _c_i64]
    lib.sbl_linear_backward_ws.restype = ctypes.c_int
    lib.sbl_linear_backward_ws.argtypes = [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i32, _c_i32, _c_i32,
                                           _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_p]
    lib.sbl_head_workspace_bytes.restype = _c_i64
    lib.sbl_head_workspace_bytes.argtypes = [_c_i64, _c_i64, _c_i64, _c_i32, _c_i32]
    sizes, tail = [_c_i64, _c_i64, _c_i64], [_c_p, _c_p, _c_p, _c_i64, _c_p]
    lib.sbl_head_ce_forward.restype = ctypes.c_int
    lib.sbl_head_ce_forward.argtypes = [_c_p, _c_i64, _c_p, _c_i32, _c_p, *sizes, *tail]
    lib.sbl_head_ce_backward.restype = ctypes.c_int
    lib.sbl_head_ce_backward.argtypes = [_c_p, _c_i64, _c_p, _c_i32, _c_p, _c_p, _c_p, _c_p, *sizes, *tail]
    lib.sbl_head_kd_forward.restype = ctypes.c_int
    lib.sbl_head_kd_forward.argtypes = [_c_p, _c_i64, _c_p, _c_i32, _c_p, _c_p, _c_i32, ctypes.c_float, *sizes, *tail]
    lib.sbl_head_kd_backward.restype = ctypes.c_int
    lib.sbl_head_kd_backward.argtypes = [_c_p, _c_i64, _c_p, _c_i32, _c_p, _c_p, _c_i32, ctypes.c_float, _c_p, _c_p,
                                         *sizes, *tail]
    c_f32, c_f64 = ctypes.c_float, ctypes.c_double
    lib.sbl_norm_forward.restype = ctypes.c_int
    lib.sbl_norm_forward.argtypes = [_c_p, _c_i32, _c_p, _c_p, _c_i64, _c_i64, c_f64, _c_i32, _c_p, _c_i32, _c_p, _c_p,
                                     _c_p, _c_p, _c_p]
    lib.sbl_norm_workspace_bytes.restype = _c_i64
    lib.sbl_norm_workspace_bytes.argtypes = [_c_i64, _c_i64]
    lib.sbl_norm_backward.restype = ctypes.c_int
    lib.sbl_norm_backward.argtypes = [_c_p, _c_i32, _c_p, _c_i32, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i32, _c_p, _c_p,
                                      _c_p, _c_p, _c_i64, _c_p]
    lib.sbl_embed_forward.restype = ctypes.c_int
    lib.sbl_embed_forward.argtypes = [_c_p, _c_p, _c_i32, _c_i64, _c_i64, _c_i64, c_f32, _c_p, _c_i32, _c_p]
    lib.sbl_embed_workspace_bytes.restype = _c_i64
    lib.sbl_embed_workspace_bytes.argtypes = [_c_i64, _c_i64, _c_i64, _c_i32]
    lib.sbl_embed_backward.restype = ctypes.c_int
    lib.sbl_embed_backward.argtypes = [_c_p, _c_p, _c_i32, _c_i64, _c_i64, _c_i64, c_f32, _c_p, _c_i32, _c_i32, _c_p,
                                       _c_i64, _c_p]
    lib.sbl_adamw_batch.restype = ctypes.c_int
    lib.sbl_adamw_batch.argtypes = [ctypes.POINTER(AdamWItem), _c_i32, c_f64, c_f64, c_f64, c_f64, _c_i64, _c_p, _c_p]


# ---------------------------------------------------------------- helpers

def _ptr(t, dtype, nbytes: int, name: str):
    """Device pointer of a contiguous tensor holding at least nbytes, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, needs {nbytes}")
    return t.data_ptr()


# The current stream's handle without the stream object (0.3 us a call, not 2.7).
# torch has the function for its own use only: where it lacks it, the public way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(func: str, status: int):
    if status != SBL_OK:
        raise SblError(func, status)


# ---------------------------------------------------------------- the C ABI, by name

def sbl_abi_version() -> int:
    return load().sbl_abi_version()


def sbl_packed_bytes(n_out: int, k: int, n: int, m: int, fmt: int) -> int:
    return load().sbl_packed_bytes(n_out, k, n, m, fmt)


def sbl_meta_bytes(n_out: int, k: int, fmt: int) -> int:
    return load().sbl_meta_bytes(n_out, k, fmt)


def sbl_workspace_bytes(n_out: int, k: int) -> int:
    return load().sbl_workspace_bytes(n_out, k)


def sbl_workspace_init(workspace, stream=None):
    """Zero-fill a whole workspace tensor (any dtype) with the library's kernel."""
    lib = load()
    nbytes = (workspace.numel() * workspace.element_size()) // 8 * 8
    _check("sbl_workspace_init",
           lib.sbl_workspace_init(_ptr(workspace, None, nbytes, "workspace"), nbytes, _stream(stream)))


_W16 = (torch.int16, torch.uint16, torch.bfloat16)


def sbl_quant_weights(w_bf16, n: int, m: int, beta, workspace, mask_bits=None, codes=None,
                      fmt: int = SBL_FMT_DENSE2, packed=None, meta=None, stream=None):
    """w_bf16: [n_out][k] BF16 (or its 16-bit patterns as int16/uint16)."""
    lib = load()
    n_out, k = w_bf16.shape
    pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt) if packed is not None else 0
    mb = n_out * k // 8
    st = lib.sbl_quant_weights(
        _ptr(w_bf16, _W16, n_out * k * 2, "w_bf16"), n_out, k, n, m,
        _ptr(beta, torch.float32, 4, "beta"),
        _ptr(mask_bits, torch.uint8, mb, "mask_bits"),
        _ptr(codes, torch.int8, n_out * k, "codes"),
        fmt, _ptr(packed, torch.uint8, max(pb, 0), "packed"),
        _ptr(meta, torch.uint8, mb, "meta") if fmt == SBL_FMT_NM else None,
        _ptr(workspace, None, lib.sbl_workspace_bytes(n_out, k), "workspace"),
        workspace.numel() * workspace.element_size() if workspace is not None else 0,
        _stream(stream))
    _check("sbl_quant_weights", st)


def _nbytes(t):
    return t.numel() * t.element_size() if t is not None else 0


def _quant_items(lib, items, n: int, m: int, fmt: int, workspaces: bool = True):
    arr = (QuantItem * len(items))()
    for i, it in enumerate(items):
        w = it["w"]
        n_out, k = w.shape
        packed = it.get("packed")
        pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt) if packed is not None else 0
        mb = n_out * k // 8
        ws = it["workspace"] if workspaces else None
        arr[i] = QuantItem(
            _ptr(w, _W16, n_out * k * 2, "w"), n_out, k, _ptr(it["beta"], torch.float32, 4, "beta"),
            _ptr(it.get("mask_bits"), torch.uint8, mb, "mask_bits"),
            _ptr(it.get("codes"), torch.int8, n_out * k, "codes"),
            _ptr(packed, torch.uint8, max(pb, 0), "packed"),
            _ptr(it.get("meta"), torch.uint8, mb, "meta") if fmt == SBL_FMT_NM else None,
            _ptr(ws, None, lib.sbl_workspace_bytes(n_out, k), "workspace") if workspaces else None,
            _nbytes(ws))
    return arr


def sbl_quant_weights_batch(items, n: int, m: int, fmt: int = SBL_FMT_DENSE2, stream=None, flags: int = 0):
    """items: sequence of dicts with keys w (BF16 [n_out][k]), beta, workspace and the
    optional outputs mask_bits, codes, packed, meta (as in sbl_quant_weights)."""
    lib = load()
    arr = _quant_items(lib, items, n, m, fmt)
    if flags:
        _check("sbl_quant_weights_batch_ex",
               lib.sbl_quant_weights_batch_ex(arr, len(items), n, m, fmt, flags, _stream(stream)))
    else:
        _check("sbl_quant_weights_batch",
               lib.sbl_quant_weights_batch(arr, len(items), n, m, fmt, _stream(stream)))


def sbl_quant_weights_batch_noalloc(items, n: int, m: int, fmt: int = SBL_FMT_DENSE2, stream=None):
    """sbl_quant_weights_batch without caller workspaces: the library's fixed
    per-GPU scratch array serves every item (a "workspace" key is ignored)."""
    lib = load()
    arr = _quant_items(lib, items, n, m, fmt, workspaces=False)
    _check("sbl_quant_weights_batch_noalloc",
           lib.sbl_quant_weights_batch_noalloc(arr, len(items), n, m, fmt, _stream(stream)))


def sbl_pack(codes, mask_bits, n: int, m: int, fmt: int, packed, meta=None, stream=None):
    lib = load()
    n_out, k = codes.shape
    pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt)
    mb = n_out * k // 8
    st = lib.sbl_pack(_ptr(codes, torch.int8, n_out * k, "codes"),
                      _ptr(mask_bits, torch.uint8, mb, "mask_bits") if fmt == SBL_FMT_NM else None,
                      n_out, k, n, m, fmt, _ptr(packed, torch.uint8, max(pb, 0), "packed"),
                      _ptr(meta, torch.uint8, mb, "meta") if fmt == SBL_FMT_NM else None,
                      _stream(stream))
    _check("sbl_pack", st)


def sbl_quant_acts(x, xq, gamma, stream=None):
    lib = load()
    m_tok, k = x.shape
    st = lib.sbl_quant_acts(_ptr(x, torch.float32, m_tok * k * 4, "x"), m_tok, k,
                            _ptr(xq, torch.int8, m_tok * k, "xq"),
                            _ptr(gamma, torch.float32, m_tok * 4, "gamma"), _stream(stream))
    _check("sbl_quant_acts", st)


def sbl_linear(packed, meta, fmt: int, n: int, m: int, beta, xq, gamma, n_out: int, y, acc=None,
               stream=None):
    lib = load()
    m_tok, k = xq.shape
    pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt) if n_out > 0 else 0
    mb = n_out * k // 8
    st = lib.sbl_linear(_ptr(packed, torch.uint8, max(pb, 0), "packed"),
                        _ptr(meta, torch.uint8, mb, "meta") if fmt == SBL_FMT_NM else None,
                        fmt, n, m, _ptr(beta, torch.float32, 4, "beta"),
                        _ptr(xq, torch.int8, m_tok * k, "xq"),
                        _ptr(gamma, torch.float32, m_tok * 4, "gamma"), m_tok, n_out, k,
                        _ptr(y, torch.float32, m_tok * n_out * 4, "y"),
                        _ptr(acc, torch.int32, m_tok * n_out * 4, "acc"), _stream(stream))
    _check("sbl_linear", st)


def sbl_workspace_bytes_grouped(n_out: int, k: int, rows_per_group: int) -> int:
    return load().sbl_workspace_bytes_grouped(n_out, k, rows_per_group)


def sbl_quant_weights_grouped(w_bf16, n: int, m: int, rows_per_group: int, beta, workspace, mask_bits=None,
                              codes=None, fmt: int = SBL_FMT_DENSE2, packed=None, meta=None, stream=None):
    """Group scales: beta fp32 [ceil(n_out / rows_per_group)], one per block of output rows."""
    lib = load()
    n_out, k = w_bf16.shape
    groups = -(-n_out // rows_per_group) if rows_per_group > 0 else 1
    pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt) if packed is not None else 0
    st = lib.sbl_quant_weights_grouped(
        _ptr(w_bf16, _W16, n_out * k * 2, "w_bf16"), n_out, k, n, m, rows_per_group,
        _ptr(beta, torch.float32, 4 * groups, "beta"),
        _ptr(mask_bits, torch.uint8, n_out * k // 8, "mask_bits"), _ptr(codes, torch.int8, n_out * k, "codes"),
        fmt, _ptr(packed, torch.uint8, max(pb, 0), "packed"),
        _ptr(meta, torch.uint8, n_out * k // 8, "meta") if fmt == SBL_FMT_NM else None,
        _ptr(workspace, None, max(lib.sbl_workspace_bytes_grouped(n_out, k, rows_per_group), 0), "workspace"),
        _nbytes(workspace), _stream(stream))
    _check("sbl_quant_weights_grouped", st)


def sbl_linear_grouped(packed, meta, fmt: int, n: int, m: int, beta, rows_per_group: int, xq, gamma, n_out: int, y,
                       acc=None, stream=None):
    lib = load()
    m_tok, k = xq.shape
    groups = -(-n_out // rows_per_group) if rows_per_group > 0 else 1
    pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt) if n_out > 0 else 0
    st = lib.sbl_linear_grouped(_ptr(packed, torch.uint8, max(pb, 0), "packed"),
                                _ptr(meta, torch.uint8, n_out * k // 8, "meta") if fmt == SBL_FMT_NM else None,
                                fmt, n, m, _ptr(beta, torch.float32, 4 * groups, "beta"), rows_per_group,
                                _ptr(xq, torch.int8, m_tok * k, "xq"), _ptr(gamma, torch.float32, m_tok * 4, "gamma"),
                                m_tok, n_out, k, _ptr(y, torch.float32, m_tok * n_out * 4, "y"),
                                _ptr(acc, torch.int32, m_tok * n_out * 4, "acc"), _stream(stream))
    _check("sbl_linear_grouped", st)


def sbl_workspace_bytes_blocked(n_out: int, k: int, rows_per_group: int, cols_per_group: int) -> int:
    return load().sbl_workspace_bytes_blocked(n_out, k, rows_per_group, cols_per_group)


def sbl_quant_weights_blocked(w_bf16, n: int, m: int, rows_per_group: int, cols_per_group: int, beta, workspace,
                              mask_bits=None, codes=None, fmt: int = SBL_FMT_DENSE2, packed=None, meta=None,
                              stream=None):
    """Block scales: beta fp32 [ceil(n_out / rows_per_group)][k // cols_per_group]."""
    lib = load()
    n_out, k = w_bf16.shape
    gr = -(-n_out // rows_per_group) if rows_per_group > 0 else 1
    gk = k // cols_per_group if cols_per_group > 0 else 1
    pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt) if packed is not None else 0
    wsb = lib.sbl_workspace_bytes_blocked(n_out, k, rows_per_group, cols_per_group)
    st = lib.sbl_quant_weights_blocked(
        _ptr(w_bf16, _W16, n_out * k * 2, "w_bf16"), n_out, k, n, m, rows_per_group, cols_per_group,
        _ptr(beta, torch.float32, 4 * gr * gk, "beta"),
        _ptr(mask_bits, torch.uint8, n_out * k // 8, "mask_bits"), _ptr(codes, torch.int8, n_out * k, "codes"),
        fmt, _ptr(packed, torch.uint8, max(pb, 0), "packed"),
        _ptr(meta, torch.uint8, n_out * k // 8, "meta") if fmt == SBL_FMT_NM else None,
        _ptr(workspace, None, max(wsb, 0), "workspace"), _nbytes(workspace), _stream(stream))
    _check("sbl_quant_weights_blocked", st)


def sbl_linear_blocked(packed, meta, fmt: int, n: int, m: int, beta, rows_per_group: int, xq, gamma, kg: int,
                       n_out: int, y, stream=None):
    """Products with block scales: beta [ceil(n_out / rows_per_group)][k // kg]."""
    lib = load()
    m_tok, k = xq.shape
    gr = -(-n_out // rows_per_group) if rows_per_group > 0 else 1
    gk = k // kg if kg > 0 else 1
    pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt) if n_out > 0 else 0
    st = lib.sbl_linear_blocked(_ptr(packed, torch.uint8, max(pb, 0), "packed"),
                                _ptr(meta, torch.uint8, n_out * k // 8, "meta") if fmt == SBL_FMT_NM else None,
                                fmt, n, m, _ptr(beta, torch.float32, 4 * gr * gk, "beta"), rows_per_group,
                                _ptr(xq, torch.int8, m_tok * k, "xq"),
                                _ptr(gamma, torch.float32, m_tok * gk * 4, "gamma"), kg, m_tok, n_out, k,
                                _ptr(y, torch.float32, m_tok * n_out * 4, "y"), _stream(stream))
    _check("sbl_linear_blocked", st)


def sbl_quant_acts_kgrouped(x, kg: int, xq, gamma, stream=None):
    """x fp32 [m_tok][k] -> xq int8 [m_tok][k], gamma fp32 [m_tok][k // kg]."""
    lib = load()
    m_tok, k = x.shape
    st = lib.sbl_quant_acts_kgrouped(_ptr(x, torch.float32, m_tok * k * 4, "x"), m_tok, k, kg,
                                     _ptr(xq, torch.int8, m_tok * k, "xq"),
                                     _ptr(gamma, torch.float32, m_tok * (k // kg) * 4, "gamma"), _stream(stream))
    _check("sbl_quant_acts_kgrouped", st)


def sbl_linear_kgrouped(packed, meta, fmt: int, n: int, m: int, beta, rows_per_group: int, xq, gamma, kg: int,
                        n_out: int, y, stream=None):
    lib = load()
    m_tok, k = xq.shape
    groups = -(-n_out // rows_per_group) if rows_per_group > 0 else 1
    pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt) if n_out > 0 else 0
    st = lib.sbl_linear_kgrouped(_ptr(packed, torch.uint8, max(pb, 0), "packed"),
                                 _ptr(meta, torch.uint8, n_out * k // 8, "meta") if fmt == SBL_FMT_NM else None,
                                 fmt, n, m, _ptr(beta, torch.float32, 4 * groups, "beta"), rows_per_group,
                                 _ptr(xq, torch.int8, m_tok * k, "xq"),
                                 _ptr(gamma, torch.float32, m_tok * (k // kg) * 4, "gamma"), kg, m_tok, n_out, k,
                                 _ptr(y, torch.float32, m_tok * n_out * 4, "y"), _stream(stream))
    _check("sbl_linear_kgrouped", st)


def sbl_backward_workspace_bytes(m_tok: int, n_out: int, k: int) -> int:
    return load().sbl_backward_workspace_bytes(m_tok, n_out, k)


def new_backward_workspace(m_tok: int, n_out: int, k: int, device="cuda"):
    """Scratch for sbl_linear_backward(..., workspace=) at these sizes (any contents)."""
    nbytes = sbl_backward_workspace_bytes(m_tok, n_out, k)
    if nbytes < 0:
        raise ValueError("unsupported shape")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def sbl_linear_backward(dy, packed, meta, fmt: int, n: int, m: int, beta, x, xq, gamma, dx=None, dw=None,
                        workspace=None, stream=None):
    """Backward of the layer (dual straight-through estimator): dy BF16 [m_tok][n_out];
    dx fp32 [m_tok][k] and/or dw fp32 [n_out][k] outputs (either may be None).  With a
    workspace (uint8, sbl_backward_workspace_bytes(m_tok, n_out, k) bytes) the call goes
    to sbl_linear_backward_ws."""
    lib = load()
    m_tok, n_out = dy.shape
    k = (xq if xq is not None else x).shape[1]
    pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt) if dx is not None else 0
    if workspace is not None:
        wsb = workspace.numel() * workspace.element_size()
        fn, extra, name = lib.sbl_linear_backward_ws, (_ptr(workspace, None, wsb, "workspace"), wsb), \
            "sbl_linear_backward_ws"
    else:
        fn, extra, name = lib.sbl_linear_backward, (), "sbl_linear_backward"
    st = fn(
        _ptr(dy, _W16, m_tok * n_out * 2, "dy"), m_tok, n_out, k,
        _ptr(packed, torch.uint8, max(pb, 0), "packed") if dx is not None else None,
        _ptr(meta, torch.uint8, n_out * k // 8, "meta") if dx is not None and fmt == SBL_FMT_NM else None,
        fmt, n, m,
        _ptr(beta, torch.float32, 4, "beta") if dx is not None else None,
        _ptr(x, torch.float32, m_tok * k * 4, "x") if dx is not None else None,
        _ptr(xq, torch.int8, m_tok * k, "xq") if dw is not None else None,
        _ptr(gamma, torch.float32, m_tok * 4, "gamma"),
        _ptr(dx, torch.float32, m_tok * k * 4, "dx"), _ptr(dw, torch.float32, n_out * k * 4, "dw"),
        *extra, _stream(stream))
    _check(name, st)


def sbl_linear_batch(items, fmt: int, n: int, m: int, stream=None):
    """items: sequence of dicts with keys packed, meta, beta, xq, gamma, n_out, y[, acc]."""
    lib = load()
    arr = (LinearItem * len(items))()
    for i, it in enumerate(items):
        m_tok, k = it["xq"].shape
        n_out = it["n_out"]
        pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt) if n_out > 0 else 0
        arr[i] = LinearItem(
            _ptr(it["packed"], torch.uint8, max(pb, 0), "packed"),
            _ptr(it.get("meta"), torch.uint8, n_out * k // 8, "meta") if fmt == SBL_FMT_NM else None,
            _ptr(it["beta"], torch.float32, 4, "beta"), _ptr(it["xq"], torch.int8, m_tok * k, "xq"),
            _ptr(it["gamma"], torch.float32, m_tok * 4, "gamma"), m_tok, n_out, k,
            _ptr(it["y"], torch.float32, m_tok * n_out * 4, "y"),
            _ptr(it.get("acc"), torch.int32, m_tok * n_out * 4, "acc"))
    _check("sbl_linear_batch", lib.sbl_linear_batch(arr, len(items), fmt, n, m, _stream(stream)))


def sbl_linear_acts_batch(x, xq, gamma, items, fmt: int, n: int, m: int, stream=None):
    """x: [m_tok][k] fp32 input; xq, gamma: its quantized form (outputs);
    items: sequence of dicts with keys packed, meta, beta, n_out, y[, acc]."""
    lib = load()
    m_tok, k = x.shape
    arr = (LinearItem * len(items))()
    for i, it in enumerate(items):
        n_out = it["n_out"]
        pb = lib.sbl_packed_bytes(n_out, k, n, m, fmt) if n_out > 0 else 0
        arr[i] = LinearItem(
            _ptr(it["packed"], torch.uint8, max(pb, 0), "packed"),
            _ptr(it.get("meta"), torch.uint8, n_out * k // 8, "meta") if fmt == SBL_FMT_NM else None,
            _ptr(it["beta"], torch.float32, 4, "beta"), None, None, m_tok, n_out, k,
            _ptr(it["y"], torch.float32, m_tok * n_out * 4, "y"),
            _ptr(it.get("acc"), torch.int32, m_tok * n_out * 4, "acc"))
    st = lib.sbl_linear_acts_batch(_ptr(x, torch.float32, m_tok * k * 4, "x"), m_tok, k,
                                   _ptr(xq, torch.int8, m_tok * k, "xq"),
                                   _ptr(gamma, torch.float32, m_tok * 4, "gamma"), arr, len(items), fmt, n, m,
                                   _stream(stream))
    _check("sbl_linear_acts_batch", st)


# ---------------------------------------------------------------- losses of the output head

def sbl_head_workspace_bytes(m_tok: int, n_vocab: int, k: int, top: int = 1, backward: bool = False) -> int:
    return load().sbl_head_workspace_bytes(m_tok, n_vocab, k, top, int(backward))


def _head_args(h, w):
    """(h pointer, row stride, w pointer, dtype, m_tok, n_vocab, k): h [m_tok][k] with rows of
    contiguous values (any row stride that is a multiple of 8), w [n_vocab][k] contiguous, both
    bfloat16 (or its 16-bit patterns as int16/uint16) or both float16, on the current GPU."""
    if not isinstance(h, torch.Tensor) or not isinstance(w, torch.Tensor):
        raise TypeError("h and w must be torch.Tensors")
    if h.dim() != 2 or w.dim() != 2:
        raise ValueError("h and w must have two dimensions")
    fp16 = h.dtype == torch.float16
    types = (torch.float16,) if fp16 else _W16
    if h.dtype not in types or w.dtype not in types:
        raise TypeError(f"h and w have dtypes {h.dtype} and {w.dtype}, expected two of {types}")
    m_tok, k = h.shape
    n_vocab, kw = w.shape
    if kw != k:
        raise ValueError(f"h has {k} features, w {kw}")
    if not h.is_cuda or h.device != w.device or h.get_device() != torch.cuda.current_device():
        raise ValueError("h and w must be on the current GPU")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    stride, step = h.stride()
    if m_tok <= 1:
        stride = k
    if step != 1 and k > 1 or stride < k:
        raise ValueError("h must have rows of contiguous values")
    return (h.data_ptr() if m_tok else None, stride, w.data_ptr(), SBL_FP16 if fp16 else SBL_BF16, m_tok, n_vocab, k)


def _teacher_args(index, teacher, m_tok: int):
    if not isinstance(index, torch.Tensor) or not isinstance(teacher, torch.Tensor):
        raise TypeError("index and teacher must be torch.Tensors")
    if index.dim() != 2 or index.shape != teacher.shape or index.shape[0] != m_tok:
        raise ValueError("index and teacher must be [m_tok][top]")
    top = index.shape[1]
    return (_ptr(index, torch.int64, m_tok * top * 8, "index"),
            _ptr(teacher, torch.float32, m_tok * top * 4, "teacher"), top)


def sbl_head_ce_forward(h, w, target, loss, lse, workspace, stream=None):
    """Cross entropy of the output head: h [m_tok][k], w [n_vocab][k] (16-bit), target int64
    [m_tok] (negative: row taken out) -> loss, lse fp32 [m_tok].  The logits are never stored."""
    head = _head_args(h, w)
    n = head[4] * 4
    _check("sbl_head_ce_forward", load().sbl_head_ce_forward(
        *head[:4], _ptr(target, torch.int64, 2 * n, "target"), *head[4:], _ptr(loss, torch.float32, n, "loss"),
        _ptr(lse, torch.float32, n, "lse"), _ptr(workspace, None, 0, "workspace"), _nbytes(workspace),
        _stream(stream)))


def sbl_head_ce_backward(h, w, target, lse, dloss, dh, dw, workspace, dlse=None, stream=None):
    """Gradients of the cross entropy: dloss (and dlse) fp32 [m_tok] -> dh [m_tok][k] and dw
    [n_vocab][k] in the type of h and w (either may be None)."""
    head = _head_args(h, w)
    m_tok, n_vocab, k = head[4:]
    n = m_tok * 4
    _check("sbl_head_ce_backward", load().sbl_head_ce_backward(
        *head[:4], _ptr(target, torch.int64, 2 * n, "target"), _ptr(lse, torch.float32, n, "lse"),
        _ptr(dloss, torch.float32, n, "dloss"), _ptr(dlse, torch.float32, n, "dlse"), m_tok, n_vocab, k,
        _ptr(dh, h.dtype, m_tok * k * 2, "dh"), _ptr(dw, w.dtype, n_vocab * k * 2, "dw"),
        _ptr(workspace, None, 0, "workspace"), _nbytes(workspace), _stream(stream)))


def sbl_head_kd_forward(h, w, index, teacher, tau: float, loss, lse, workspace, stream=None):
    """Distillation from a teacher's top logits: index int64, teacher fp32 [m_tok][top]
    (negative index: no entry), tau the temperature -> loss, lse fp32 [m_tok]."""
    head = _head_args(h, w)
    n = head[4] * 4
    _check("sbl_head_kd_forward", load().sbl_head_kd_forward(
        *head[:4], *_teacher_args(index, teacher, head[4]), tau, *head[4:], _ptr(loss, torch.float32, n, "loss"),
        _ptr(lse, torch.float32, n, "lse"), _ptr(workspace, None, 0, "workspace"), _nbytes(workspace),
        _stream(stream)))


def sbl_head_kd_backward(h, w, index, teacher, tau: float, lse, dloss, dh, dw, workspace, stream=None):
    """Gradients of the distillation loss: dloss fp32 [m_tok] -> dh [m_tok][k] and dw
    [n_vocab][k] in the type of h and w (either may be None)."""
    head = _head_args(h, w)
    m_tok, n_vocab, k = head[4:]
    _check("sbl_head_kd_backward", load().sbl_head_kd_backward(
        *head[:4], *_teacher_args(index, teacher, m_tok), tau, _ptr(lse, torch.float32, m_tok * 4, "lse"),
        _ptr(dloss, torch.float32, m_tok * 4, "dloss"), m_tok, n_vocab, k, _ptr(dh, h.dtype, m_tok * k * 2, "dh"),
        _ptr(dw, w.dtype, n_vocab * k * 2, "dw"), _ptr(workspace, None, 0, "workspace"), _nbytes(workspace),
        _stream(stream)))


# ---------------------------------------------------------------- norm, embedding, AdamW

_TYPES = {torch.bfloat16: SBL_BF16, torch.float16: SBL_FP16, torch.float32: SBL_FP32}


def _type(t, name: str) -> int:
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(_TYPES)}") from None


def _here(t, dtype, shape, name: str, device: int):
    """Device pointer of a contiguous tensor of this shape on the current GPU (`device`), or None."""
    if t is None:
        return None
    _tensor(t, name)
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the current GPU")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _tensor(t, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")


def _rows(t, name: str):
    _tensor(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return t.shape


def _scratch(t, device: int):
    """(pointer, bytes) of a workspace."""
    if t is None:
        return None, 0
    return _here(t, None, t.shape, "workspace", device), _nbytes(t)


def sbl_norm_forward(x, weight=None, bias=None, eps: float = 1e-5, center: bool = True, y=None, xq=None, gamma=None,
                     mean=None, rstd=None, stream=None):
    """Layer norm (center) or RMS norm of the rows of x [m_tok][k] -> y (x's type, or one of them fp32) and/or its
    int8 codes xq with gamma; mean, rstd fp32 [m_tok] for the backward.  Every output may be None."""
    m_tok, k = rows = _rows(x, "x")
    f32, device, row, col = torch.float32, torch.cuda.current_device(), (m_tok,), (k,)
    st = load().sbl_norm_forward(
        _here(x, None, rows, "x", device), _type(x, "x"), _here(weight, f32, col, "weight", device),
        _here(bias, f32, col, "bias", device), m_tok, k, eps, center, _here(y, None, rows, "y", device),
        _type(y if y is not None else x, "y"), _here(xq, torch.int8, rows, "xq", device),
        _here(gamma, f32, row, "gamma", device), _here(mean, f32, row, "mean", device),
        _here(rstd, f32, row, "rstd", device), _stream(stream))
    if st != SBL_OK:
        raise SblError("sbl_norm_forward", st)


def sbl_norm_workspace_bytes(m_tok: int, k: int) -> int:
    return load().sbl_norm_workspace_bytes(m_tok, k)


def sbl_norm_backward(dy, x, mean, rstd, weight, dx, dweight, dbias, workspace, center: bool = True, stream=None):
    """Gradients of the norm from dy [m_tok][k] (x's type, or one of them fp32): dx in x's type, dweight and dbias fp32 [k]
    (each may be None).  mean may be None where not centered."""
    m_tok, k = rows = _rows(x, "x")
    f32, device, row, col = torch.float32, torch.cuda.current_device(), (m_tok,), (k,)
    _check("sbl_norm_backward", load().sbl_norm_backward(
        _here(dy, None, rows, "dy", device), _type(dy, "dy"), _here(x, None, rows, "x", device), _type(x, "x"),
        _here(mean, f32, row, "mean", device), _here(rstd, f32, row, "rstd", device),
        _here(weight, f32, col, "weight", device), m_tok, k, center, _here(dx, x.dtype, rows, "dx", device),
        _here(dweight, f32, col, "dweight", device), _here(dbias, f32, col, "dbias", device), *_scratch(workspace, device),
        _stream(stream)))


def _ids(ids):
    _tensor(ids, "ids")
    device = torch.cuda.current_device()
    return _here(ids, torch.int64, ids.shape, "ids", device), ids.numel(), device


def sbl_embed_forward(ids, table, out, scale: float = 1.0, stream=None):
    """out[t] = scale * table[ids[t]]: ids int64 of any shape, table [n_vocab][k], out [ids' shape][k] in the
    table's type (or one of them fp32).  A negative id gives zeros, an id past the table NaNs."""
    n_vocab, k = rows = _rows(table, "table")
    at, m_tok, device = _ids(ids)
    _check("sbl_embed_forward", load().sbl_embed_forward(
        at, _here(table, None, rows, "table", device), _type(table, "table"), m_tok, n_vocab, k, scale,
        _here(out, None, (*ids.shape, k), "out", device), _type(out, "out"), _stream(stream)))


def sbl_embed_workspace_bytes(m_tok: int, n_vocab: int, k: int, dtype=torch.bfloat16) -> int:
    """dtype: of the gradient that comes in."""
    if dtype not in _TYPES:
        raise TypeError(f"dtype is {dtype}, expected one of {tuple(_TYPES)}")
    return load().sbl_embed_workspace_bytes(m_tok, n_vocab, k, _TYPES[dtype])


def sbl_embed_backward(ids, dout, dtable, workspace, scale: float = 1.0, add: bool = False, stream=None):
    """Gradient of the table from dout [ids' shape][k] (the table's type, or one of them fp32): written to dtable
    [n_vocab][k], or added to what it holds."""
    n_vocab, k = rows = _rows(dtable, "dtable")
    at, m_tok, device = _ids(ids)
    _check("sbl_embed_backward", load().sbl_embed_backward(
        at, _here(dout, None, (*ids.shape, k), "dout", device), _type(dout, "dout"), m_tok, n_vocab, k, scale,
        _here(dtable, None, rows, "dtable", device), _type(dtable, "dtable"), add, *_scratch(workspace, device),
        _stream(stream)))


class AdamWItems:
    """The tensors of an AdamW step, checked once and kept alive: a sequence of dicts with keys
      w             weights, any shape, contiguous: bfloat16, float16 or float32 (updated in place)
      w_low         int16, of BF16 masters: the low bits of an fp32 weight (split_master), or absent
      g             gradient, bfloat16, float16 or float32
      m, v          states: both float32, or both float8_e4m3fn (or their bytes as uint8) with
      m_scale, v_scale  float32, one for each 256 values
      lr_scale, weight_decay  numbers (1 and 0 if absent)
    of as many values as w each."""

    def __init__(self, tensors):
        self.tensors = [dict(t) for t in tensors]
        if not self.tensors:
            raise ValueError("no tensors")
        self.device = None
        self.array = (AdamWItem * len(self.tensors))()
        for i, t in enumerate(self.tensors):
            for name in ("w", "g", "m", "v"):
                if name not in t:
                    raise ValueError(f"tensor {i} has no {name}")
                _tensor(t[name], name)
            w, n = t["w"], t["w"].numel()
            self._on_device(w, "w")
            small = t["m"].dtype != torch.float32
            state = (torch.float8_e4m3fn, torch.uint8) if small else torch.float32
            scales = 4 * (-(-n // 256)) if small else 0
            for name in ("m", "v", "w_low", "m_scale", "v_scale"):
                if t.get(name) is not None:
                    self._on_device(t[name], name)
            if t["m"].numel() != n or t["v"].numel() != n:
                raise ValueError(f"m and v have {t['m'].numel()} and {t['v'].numel()} values, w {n}")
            self.array[i] = AdamWItem(
                _ptr(w, None, 0, "w"), _ptr(t.get("w_low"), torch.int16, 2 * n, "w_low"), None,
                _ptr(t["m"], state, n, "m"), _ptr(t["v"], state, n, "v"),
                _ptr(t.get("m_scale"), torch.float32, scales, "m_scale") if small else None,
                _ptr(t.get("v_scale"), torch.float32, scales, "v_scale") if small else None, n, _type(w, "w"), 0,
                8 if small else 32, float(t.get("lr_scale", 1.0)), float(t.get("weight_decay", 0.0)))
            self.set_gradient(i, t["g"])

    def _on_device(self, t, name: str):
        _tensor(t, name)
        if not t.is_cuda or self.device not in (None, t.device):
            raise ValueError(f"{name} must be on the GPU that the first tensor is on")
        self.device = t.device

    def set_gradient(self, i: int, g):
        """Tensor i's gradient of the next steps."""
        t, item = self.tensors[i], self.array[i]
        self._on_device(g, "g")
        if g.numel() != item.n:
            raise ValueError(f"g has {g.numel()} values, w {item.n}")
        item.g, item.g_dtype = _ptr(g, None, 0, "g"), _type(g, "g")
        t["g"] = g


def sbl_adamw_batch(items, lr: float, beta1: float, beta2: float, eps: float, step: int, schedule=None, stream=None):
    """One AdamW step of every tensor of `items` (an AdamWItems, or a sequence of its dicts).  schedule: float32
    [5] on the GPU (adamw_schedule), read in place of lr and step when the step runs."""
    if not isinstance(items, AdamWItems):
        items = AdamWItems(items)
    device = torch.cuda.current_device()
    if items.device.index != device:
        raise ValueError("the tensors must be on the current GPU")
    _check("sbl_adamw_batch", load().sbl_adamw_batch(
        items.array, len(items.tensors), lr, beta1, beta2, eps, step,
        _here(schedule, torch.float32, (5,), "schedule", device), _stream(stream)))


# ---------------------------------------------------------------- allocating conveniences

def new_workspace(n_out: int, k: int, device="cuda"):
    """A workspace for n_out x k matrices (reusable, call after call; any contents)."""
    nbytes = sbl_workspace_bytes(n_out, k)
    if nbytes < 0:
        raise ValueError("unsupported shape")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def quant_weights(w_bf16, n: int, m: int, fmt: int = SBL_FMT_DENSE2, want_codes: bool = False,
                  workspace=None, stream=None):
    """Allocate outputs and run sbl_quant_weights; returns a dict of device tensors."""
    n_out, k = w_bf16.shape
    dev = w_bf16.device
    out = {"beta": torch.empty(1, dtype=torch.float32, device=dev),
           "mask": torch.empty((n_out, k // 8), dtype=torch.uint8, device=dev)}
    pb = sbl_packed_bytes(n_out, k, n, m, fmt)
    if pb < 0:
        raise ValueError("unsupported shape or pattern")
    out["packed"] = torch.empty(pb, dtype=torch.uint8, device=dev)
    out["meta"] = torch.empty((n_out, k // 8), dtype=torch.uint8, device=dev) if fmt == SBL_FMT_NM else None
    out["codes"] = torch.empty((n_out, k), dtype=torch.int8, device=dev) if want_codes else None
    ws = workspace if workspace is not None else new_workspace(n_out, k, dev)
    sbl_quant_weights(w_bf16, n, m, out["beta"], ws, mask_bits=out["mask"], codes=out["codes"],
                      fmt=fmt, packed=out["packed"], meta=out["meta"], stream=stream)
    return out


def quant_acts(x, stream=None):
    m_tok, k = x.shape
    xq = torch.empty((m_tok, k), dtype=torch.int8, device=x.device)
    gamma = torch.empty(m_tok, dtype=torch.float32, device=x.device)
    sbl_quant_acts(x, xq, gamma, stream=stream)
    return xq, gamma


def linear(packed, meta, fmt, n, m, beta, xq, gamma, n_out, want_acc=False, stream=None):
    m_tok = xq.shape[0]
    y = torch.empty((m_tok, n_out), dtype=torch.float32, device=xq.device)
    acc = torch.empty((m_tok, n_out), dtype=torch.int32, device=xq.device) if want_acc else None
    sbl_linear(packed, meta, fmt, n, m, beta, xq, gamma, n_out, y, acc, stream=stream)
    return y, acc


def new_head_workspace(m_tok: int, n_vocab: int, k: int, top: int = 1, backward: bool = False, device="cuda"):
    """Scratch for the head calls at these sizes (any contents)."""
    nbytes = sbl_head_workspace_bytes(m_tok, n_vocab, k, top, backward)
    if nbytes < 0:
        raise ValueError("unsupported shape")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _torch_stream(stream):
    """A caller's stream as torch knows it: what a call allocates under it comes from, and
    goes back to, that stream's memory."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream)) if int(stream) != 0 else torch.cuda.default_stream()


def _new_scratch(lib, head, top: int, backward: int, device):
    """A workspace for one call on the current stream."""
    nbytes = lib.sbl_head_workspace_bytes(*head[4:], top, backward)
    return torch.empty(max(nbytes, 0), dtype=torch.uint8, device=device), nbytes


def head_ce(h, w, target, workspace=None, stream=None):
    """Allocate outputs (and a workspace) and run sbl_head_ce_forward; returns (loss, lse)."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return head_ce(h, w, target, workspace)
    lib, head = load(), _head_args(h, w)
    m_tok, device = head[4], h.device
    scratch, nbytes = (workspace, _nbytes(workspace)) if workspace is not None else \
        _new_scratch(lib, head, 1, 0, device)
    loss = torch.empty(m_tok, dtype=torch.float32, device=device)
    lse = torch.empty(m_tok, dtype=torch.float32, device=device)
    _check("sbl_head_ce_forward", lib.sbl_head_ce_forward(
        *head[:4], _ptr(target, torch.int64, 8 * m_tok, "target"), *head[4:], loss.data_ptr(), lse.data_ptr(),
        _ptr(scratch, None, 0, "workspace"), nbytes, _stream(None)))
    return loss, lse


def head_ce_backward(h, w, target, lse, dloss, dlse=None, workspace=None, stream=None):
    """Allocate outputs (and a workspace) and run sbl_head_ce_backward; returns (dh, dw)."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return head_ce_backward(h, w, target, lse, dloss, dlse, workspace)
    if workspace is None:
        workspace, _ = _new_scratch(load(), _head_args(h, w), 1, 1, h.device)
    dh, dw = torch.empty(h.shape, dtype=h.dtype, device=h.device), torch.empty_like(w)
    sbl_head_ce_backward(h, w, target, lse, dloss, dh, dw, workspace, dlse=dlse)
    return dh, dw


def head_kd(h, w, index, teacher, tau: float, workspace=None, stream=None):
    """Allocate outputs (and a workspace) and run sbl_head_kd_forward; returns (loss, lse)."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return head_kd(h, w, index, teacher, tau, workspace)
    lib, head = load(), _head_args(h, w)
    m_tok, device = head[4], h.device
    entries = _teacher_args(index, teacher, m_tok)
    scratch, nbytes = (workspace, _nbytes(workspace)) if workspace is not None else \
        _new_scratch(lib, head, entries[2], 0, device)
    loss = torch.empty(m_tok, dtype=torch.float32, device=device)
    lse = torch.empty(m_tok, dtype=torch.float32, device=device)
    _check("sbl_head_kd_forward", lib.sbl_head_kd_forward(
        *head[:4], *entries, tau, *head[4:], loss.data_ptr(), lse.data_ptr(), _ptr(scratch, None, 0, "workspace"),
        nbytes, _stream(None)))
    return loss, lse


def head_kd_backward(h, w, index, teacher, tau: float, lse, dloss, workspace=None, stream=None):
    """Allocate outputs (and a workspace) and run sbl_head_kd_backward; returns (dh, dw)."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return head_kd_backward(h, w, index, teacher, tau, lse, dloss, workspace)
    if workspace is None:
        head = _head_args(h, w)
        workspace, _ = _new_scratch(load(), head, _teacher_args(index, teacher, head[4])[2], 1, h.device)
    dh, dw = torch.empty(h.shape, dtype=h.dtype, device=h.device), torch.empty_like(w)
    sbl_head_kd_backward(h, w, index, teacher, tau, lse, dloss, dh, dw, workspace)
    return dh, dw


def _like(x, dtype, name: str):
    """The output type: x's unless another is asked for (one of the two float32)."""
    if dtype is None or dtype is x.dtype:
        return x.dtype
    if dtype not in _TYPES or (dtype is not torch.float32 and x.dtype is not torch.float32):
        raise TypeError(f"{name} must be {x.dtype} or torch.float32")
    return dtype


def _norm_out(x, weight, bias, eps, center, y, quant: bool):
    """Run sbl_norm_forward on outputs made here, which need no checks: (xq or None, [mean, rstd, and with xq gamma])."""
    m_tok, k = rows = _rows(x, "x")
    device, where = torch.cuda.current_device(), x.device
    at, x_type = _here(x, None, rows, "x", device), _type(x, "x")
    w, b = _here(weight, torch.float32, (k,), "weight", device), _here(bias, torch.float32, (k,), "bias", device)
    stat = torch.empty((3 if quant else 2, m_tok), dtype=torch.float32, device=where)
    xq = torch.empty(rows, dtype=torch.int8, device=where) if quant else None
    p = stat.data_ptr()
    st = load().sbl_norm_forward(
        at, x_type, w, b, m_tok, k, eps, center, y.data_ptr() if y is not None else None,
        _TYPES[y.dtype] if y is not None else x_type, xq.data_ptr() if quant else None, p + 8 * m_tok if quant else None,
        p, p + 4 * m_tok, _stream(None))
    if st != SBL_OK:
        raise SblError("sbl_norm_forward", st)
    return xq, stat


def norm(x, weight=None, bias=None, eps: float = 1e-5, center: bool = True, dtype=None, stream=None):
    """Allocate outputs and run sbl_norm_forward; returns (y, mean, rstd), y in x's type unless another
    is asked for."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return norm(x, weight, bias, eps, center, dtype)
    y = torch.empty(_rows(x, "x"), dtype=_like(x, dtype, "dtype"), device=x.device)
    mean, rstd = _norm_out(x, weight, bias, eps, center, y, False)[1]
    return y, mean, rstd


def norm_quant(x, weight=None, bias=None, eps: float = 1e-5, center: bool = True, dtype=None, want_y: bool = True,
               stream=None):
    """Allocate outputs and run sbl_norm_forward with the activation quantizer; returns (xq, gamma, y, mean, rstd):
    what linear takes, and what the backward of both takes (y None unless wanted)."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return norm_quant(x, weight, bias, eps, center, dtype, want_y)
    y = torch.empty(_rows(x, "x"), dtype=_like(x, dtype, "dtype"), device=x.device) if want_y else None
    xq, stat = _norm_out(x, weight, bias, eps, center, y, True)
    mean, rstd, gamma = stat
    return xq, gamma, y, mean, rstd


def new_norm_workspace(m_tok: int, k: int, device="cuda"):
    """Scratch for sbl_norm_backward at these sizes (any contents)."""
    nbytes = sbl_norm_workspace_bytes(m_tok, k)
    if nbytes < 0:
        raise ValueError("unsupported shape")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def norm_backward(dy, x, mean, rstd, weight=None, want_bias: bool = False, center: bool = True, workspace=None,
                  stream=None):
    """Allocate outputs (and a workspace) and run sbl_norm_backward; returns (dx, dweight, dbias), dbias None
    unless wanted.  dweight is that of a weight of ones where weight is None."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return norm_backward(dy, x, mean, rstd, weight, want_bias, center, workspace)
    m_tok, k = _rows(x, "x")
    if workspace is None:
        workspace = new_norm_workspace(m_tok, k, x.device)
    dx = torch.empty((m_tok, k), dtype=x.dtype, device=x.device)
    dweight = torch.empty(k, dtype=torch.float32, device=x.device)
    dbias = torch.empty(k, dtype=torch.float32, device=x.device) if want_bias else None
    sbl_norm_backward(dy, x, mean, rstd, weight, dx, dweight, dbias, workspace, center=center)
    return dx, dweight, dbias


def embed(ids, table, scale: float = 1.0, dtype=None, stream=None):
    """Allocate the output and run sbl_embed_forward; returns rows of the table's type unless another is
    asked for."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return embed(ids, table, scale, dtype)
    _tensor(ids, "ids")
    _, k = _rows(table, "table")
    out = torch.empty((*ids.shape, k), dtype=_like(table, dtype, "dtype"), device=table.device)
    sbl_embed_forward(ids, table, out, scale)
    return out


def new_embed_workspace(m_tok: int, n_vocab: int, k: int, dtype=torch.bfloat16, device="cuda"):
    """Scratch for sbl_embed_backward at these sizes (any contents); dtype: of the gradient that comes in."""
    nbytes = sbl_embed_workspace_bytes(m_tok, n_vocab, k, dtype)
    if nbytes < 0:
        raise ValueError("unsupported shape")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def embed_backward(ids, dout, n_vocab: int, scale: float = 1.0, dtype=None, add_to=None, workspace=None, stream=None):
    """Allocate outputs (and a workspace) and run sbl_embed_backward; returns the table's gradient [n_vocab][k] in
    dtype (dout's unless given), or add_to with the gradient added."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream)):
            return embed_backward(ids, dout, n_vocab, scale, dtype, add_to, workspace)
    for t, name in ((ids, "ids"), (dout, "dout"), (add_to, "add_to")):
        if t is not None or name != "add_to":
            _tensor(t, name)
    if dout.dim() == 0:
        raise ValueError("dout must have a row for each id")
    k = dout.shape[-1]
    if add_to is not None and tuple(add_to.shape) != (n_vocab, k):
        raise ValueError(f"add_to has shape {tuple(add_to.shape)}, expected {(n_vocab, k)}")
    out = add_to if add_to is not None else \
        torch.empty((n_vocab, k), dtype=dtype if dtype is not None else dout.dtype, device=dout.device)
    if workspace is None:
        workspace = new_embed_workspace(ids.numel(), n_vocab, k, dout.dtype, dout.device)
    sbl_embed_backward(ids, dout, out, workspace, scale, add=add_to is not None)
    return out


def split_master(w32):
    """An fp32 weight as BF16 master and int16 low bits: (w, w_low), nearest BF16, ties away from zero; a NaN as the
    BF16 0x7FC0 and 0."""
    _tensor(w32, "w32")
    if w32.dtype != torch.float32:
        raise TypeError(f"w32 has dtype {w32.dtype}, expected torch.float32")
    bits = w32.contiguous().view(torch.int32).masked_fill(torch.isnan(w32), 0x7FC00000)
    high = (bits + 0x8000) >> 16
    return high.to(torch.int16).view(torch.bfloat16), (bits - (high << 16)).to(torch.int16)


def join_master(w, w_low):
    """The fp32 weight that a BF16 master and its low bits are."""
    for t, dtype, name in ((w, torch.bfloat16, "w"), (w_low, torch.int16, "w_low")):
        _tensor(t, name)
        if t.dtype != dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if w.shape != w_low.shape:
        raise ValueError(f"w has shape {tuple(w.shape)}, w_low {tuple(w_low.shape)}")
    return ((w.view(torch.int16).to(torch.int32) << 16) + w_low.to(torch.int32)).view(torch.float32)


def adamw_state(w, bits: int = 32):
    """The states of w before the first step, as keys of an AdamWItems dict: m and v, in 8 bits with their scales."""
    _tensor(w, "w")
    n, device = w.numel(), w.device
    if bits == 32:
        return {name: torch.zeros(n, dtype=torch.float32, device=device) for name in ("m", "v")}
    if bits != 8:
        raise ValueError("bits must be 8 or 32")
    state = {name: torch.zeros(n, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for name in ("m", "v")}
    state.update({name: torch.zeros(-(-n // 256), dtype=torch.float32, device=device) for name in ("m_scale", "v_scale")})
    return state


def adamw_schedule(lr: float, beta1: float, beta2: float, step: int, factor: float = 1.0):
    """The five numbers of a step's schedule, as a float32 tensor on the host."""
    if step < 1:
        raise ValueError("steps are counted from 1")
    return torch.tensor([lr, 1.0 / (1.0 - beta1 ** step), (1.0 - beta2 ** step) ** -0.5, factor,
                         float(step % (1 << 24))], dtype=torch.float32)
