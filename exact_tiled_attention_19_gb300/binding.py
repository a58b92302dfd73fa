"""ctypes binding of the C ABI in ``include/etattn.h``.

The functions ``attn_fwd``, ``attn_fwd_ex``, ``attn_bwd``, ``attn_bwd_workspace_size``,
``attn_fwd_splitkv``, ``attn_fwd_splitkv_noalloc``,
``attn_fwd_splitkv_workspace_size``, ``attn_fwd_splitkv_plan``,
``attn_fwd_global``,
``attn_fwd_varlen_splitkv``, ``attn_fwd_varlen_splitkv_workspace_size``,
``attn_fwd_varlen_splitkv_plan``,
``attn_fwd_varlen_global``,
``attn_fwd_varlen``, ``attn_fwd_varlen_ex``, ``attn_fwd_host``, ``attn_fwd_varlen_host``,
``attn_fwd_varlen_host_plan``,
``attn_qk_norm_rope``, ``attn_qk_norm_rope_bwd``, ``attn_qk_norm_rope_bwd_workspace_size``,
``attn_paged_append``, ``attn_fwd_paged``, ``attn_fwd_paged_workspace_size``, ``attn_fwd_paged_plan``,
``etattn_status_string``, ``etattn_last_cuda_error``,
``etattn_read_device_status``, ``etattn_selftest_wait_timeout`` and
``etattn_version`` have the C names and
arguments (pointers as ints).  The helpers ``attention`` and
``attention_varlen`` (and the others below) marshal torch CUDA tensors (output
allocation, strides, the current stream) and call them; every step of the computation runs in the
library's kernels.  There is no fallback: if the
library is missing or cannot be loaded, an error is raised.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
import threading

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libetattn.so")

ETATTN_F16 = 0
ETATTN_BF16 = 1
STATUS_NAMES = {
    0: "ETATTN_OK", 1: "ETATTN_ERR_NULL_PTR", 2: "ETATTN_ERR_BAD_DTYPE", 3: "ETATTN_ERR_BAD_SHAPE",
    4: "ETATTN_ERR_BAD_HEADS", 5: "ETATTN_ERR_BAD_STRIDE", 6: "ETATTN_ERR_BAD_ALIGN", 7: "ETATTN_ERR_ALIAS",
    8: "ETATTN_ERR_BAD_SCALE", 9: "ETATTN_ERR_BAD_SEQLENS", 10: "ETATTN_ERR_LAUNCH", 11: "ETATTN_ERR_DEVICE",
    12: "ETATTN_ERR_NO_DEVICE", 13: "ETATTN_ERR_BAD_INDEX",
}
globals().update({name: code for code, name in STATUS_NAMES.items()})


class EtattnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = f"{where}: {STATUS_NAMES.get(code, code)} ({etattn_status_string(code)})"
        if code == 10:
            msg += f"; cudaError={etattn_last_cuda_error()}"
        super().__init__(msg)


_lib = None
_lock = threading.Lock()
_i64p = ctypes.POINTER(ctypes.c_int64)
_i32p = ctypes.POINTER(ctypes.c_int32)
_vp = ctypes.c_void_p
_int = ctypes.c_int


def load_library(path: str | None = None):
    """Load libetattn.so (building it first when it is absent and nvcc is
    available).  Raises OSError / RuntimeError when it cannot be loaded."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or LIB_PATH
        if not os.path.exists(path):
            from . import build_lib
            path = build_lib.build()
        lib = ctypes.CDLL(path)
        lib.attn_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _int, _int, _i64p, _int,
                                 ctypes.c_float, _vp]
        lib.attn_fwd.restype = _int
        lib.attn_fwd_ex.argtypes = [_vp] * 5 + [_int] * 7 + [_i64p] + [_int] * 3 + [ctypes.c_float, _vp]
        lib.attn_fwd_ex.restype = _int
        lib.attn_fwd_varlen_ex.argtypes = [_vp] * 9 + [_int] * 9 + [_i64p] + [_int] * 3 + [ctypes.c_float, _vp]
        lib.attn_fwd_varlen_ex.restype = _int
        lib.attn_fwd_varlen_splitkv.argtypes = ([_vp] * 9 + [_int] * 9 + [_i64p] + [_int] * 3 +
                                                [ctypes.c_float, _int, _vp, ctypes.c_size_t, _vp])
        lib.attn_fwd_varlen_splitkv.restype = _int
        lib.attn_fwd_varlen_splitkv_plan.argtypes = [_int] * 5 + [ctypes.POINTER(_int)]
        lib.attn_fwd_varlen_splitkv_plan.restype = _int
        lib.attn_fwd_varlen_splitkv_workspace_size.argtypes = [_int] * 4
        lib.attn_fwd_varlen_splitkv_workspace_size.restype = ctypes.c_size_t
        lib.attn_fwd_varlen_global.argtypes = [_vp] * 9 + [_int] * 9 + [_i64p] + [_int] * 4 + [ctypes.c_float, _vp]
        lib.attn_fwd_varlen_global.restype = _int
        lib.attn_fwd_splitkv.argtypes = ([_vp] * 5 + [_int] * 7 + [_i64p] + [_int] * 3 + [ctypes.c_float, _int, _vp,
                                         ctypes.c_size_t, _vp])
        lib.attn_fwd_splitkv.restype = _int
        lib.attn_bwd.argtypes = [_vp] * 9 + [_int] * 7 + [_i64p] + [_int] * 3 + [ctypes.c_float, _vp, ctypes.c_size_t,
                                                                                   _vp]
        lib.attn_bwd.restype = _int
        lib.attn_bwd_workspace_size.argtypes = [_int] * 4
        lib.attn_bwd_workspace_size.restype = ctypes.c_size_t
        lib.attn_fwd_splitkv_noalloc.argtypes = ([_vp] * 5 + [_int] * 7 + [_i64p] + [_int] * 3 +
                                                 [ctypes.c_float, _int, _vp])
        lib.attn_fwd_splitkv_noalloc.restype = _int
        lib.attn_fwd_splitkv_workspace_size.argtypes = [_int] * 5
        lib.attn_fwd_splitkv_workspace_size.restype = ctypes.c_size_t
        lib.attn_fwd_splitkv_plan.argtypes = [_int] * 5 + [ctypes.POINTER(_int)]
        lib.attn_fwd_splitkv_plan.restype = _int
        lib.attn_fwd_global.argtypes = [_vp] * 5 + [_int] * 7 + [_i64p] + [_int] * 4 + [ctypes.c_float, _vp]
        lib.attn_fwd_global.restype = _int
        lib.attn_fwd_varlen.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _int, _int,
                                        _int, _i64p, _int, ctypes.c_float, _vp]
        lib.attn_fwd_varlen.restype = _int
        lib.attn_fwd_host.argtypes = [_vp] * 10 + [_int] * 7 + [ctypes.c_float, _vp]
        lib.attn_fwd_host.restype = _int
        lib.attn_fwd_varlen_host.argtypes = [_vp] * 12 + [_int] * 8 + [ctypes.c_float, _vp]
        lib.attn_fwd_varlen_host.restype = _int
        lib.attn_fwd_varlen_host_plan.argtypes = [_vp, _int, _int, ctypes.POINTER(ctypes.c_int32)]
        lib.attn_fwd_varlen_host_plan.restype = _int
        lib.attn_qk_norm_rope.argtypes = [_vp] * 9 + [_int] * 5 + [ctypes.c_char_p] + [_int] * 3 + [ctypes.c_float, _vp]
        lib.attn_qk_norm_rope.restype = _int
        lib.attn_qk_norm_rope_bwd.argtypes = ([_vp] * 13 + [_int] * 5 + [ctypes.c_char_p] + [_int] * 3 +
                                              [ctypes.c_float, _vp, ctypes.c_size_t, _vp])
        lib.attn_qk_norm_rope_bwd.restype = _int
        lib.attn_qk_norm_rope_bwd_workspace_size.argtypes = [_int] * 4
        lib.attn_qk_norm_rope_bwd_workspace_size.restype = ctypes.c_size_t
        lib.attn_paged_append.argtypes = ([_vp] * 13 + [_int] * 6 + [ctypes.c_char_p] + [_int] * 3 + [ctypes.c_int64] +
                                          [_int] * 3 + [ctypes.c_float, _vp])
        lib.attn_paged_append.restype = _int
        lib.attn_fwd_paged.argtypes = ([_vp] * 8 + [_int] * 7 + [ctypes.c_char_p] + [_int] * 3 + [ctypes.c_int64] + [_int] * 3 +
                                       [ctypes.c_float, _int, _vp, ctypes.c_size_t, _vp])
        lib.attn_fwd_paged.restype = _int
        lib.attn_fwd_paged_workspace_size.argtypes = [_int] * 5
        lib.attn_fwd_paged_workspace_size.restype = ctypes.c_size_t
        lib.attn_fwd_paged_plan.argtypes = [_int] * 6 + [ctypes.POINTER(_int), ctypes.POINTER(ctypes.c_size_t)]
        lib.attn_fwd_paged_plan.restype = _int
        lib.etattn_status_string.argtypes = [_int]
        lib.etattn_status_string.restype = ctypes.c_char_p
        lib.etattn_last_cuda_error.argtypes = []
        lib.etattn_last_cuda_error.restype = _int
        lib.etattn_read_device_status.argtypes = [ctypes.POINTER(_int), _int, _vp]
        lib.etattn_read_device_status.restype = _int
        lib.etattn_version.argtypes = []
        lib.etattn_version.restype = _int
        lib.etattn_selftest_wait_timeout.argtypes = [_int, _vp]
        lib.etattn_selftest_wait_timeout.restype = _int
        _lib = lib
        return lib


# ---------------------------------------------------------------- raw C entry points

def _strides_arg(strides):
    arr = (ctypes.c_int64 * len(strides))(*[int(s) for s in strides])
    return arr


def attn_fwd(q, k, v, o, lse, B, Hq, Hkv, N, D, dtype, strides, causal, scale, stream):
    """C ``attn_fwd``: pointers as ints (0 for NULL), ``strides`` 16 ints."""
    lib = load_library()
    return lib.attn_fwd(q or None, k or None, v or None, o or None, lse or None, B, Hq, Hkv, N, D, dtype,
                        _strides_arg(strides), causal, scale, stream or None)


def attn_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, dtype, strides, causal, window_left, window_right, scale,
                stream):
    """C ``attn_fwd_ex``: pointers as ints (0 for NULL), ``strides`` 16 ints."""
    lib = load_library()
    return lib.attn_fwd_ex(q or None, k or None, v or None, o or None, lse or None, B, Hq, Hkv, Nq, Nk, D, dtype,
                           _strides_arg(strides), causal, window_left, window_right, scale, stream or None)


def attn_fwd_splitkv(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, dtype, strides, causal, window_left, window_right, scale,
                     num_splits, workspace, workspace_bytes, stream):
    """C ``attn_fwd_splitkv``: pointers as ints (0 for NULL), ``strides`` 16 ints."""
    lib = load_library()
    return lib.attn_fwd_splitkv(q or None, k or None, v or None, o or None, lse or None, B, Hq, Hkv, Nq, Nk, D,
                                dtype, _strides_arg(strides), causal, window_left, window_right, scale, num_splits,
                                workspace or None, workspace_bytes, stream or None)


def attn_fwd_global(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, dtype, strides, causal, window_left, window_right,
                    num_global, scale, stream):
    """C ``attn_fwd_global``: pointers as ints (0 for NULL), ``strides`` 16 ints."""
    lib = load_library()
    return lib.attn_fwd_global(q or None, k or None, v or None, o or None, lse or None, B, Hq, Hkv, Nq, Nk, D, dtype,
                               _strides_arg(strides), causal, window_left, window_right, num_global, scale,
                               stream or None)


def attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, Nq, Nk, D, dtype, strides, causal, window_left,
             window_right, scale, workspace, workspace_bytes, stream):
    """C ``attn_bwd``: pointers as ints (0 for NULL), ``strides`` 32 ints."""
    lib = load_library()
    return lib.attn_bwd(q or None, k or None, v or None, o or None, lse or None, dout or None, dq or None, dk or None,
                        dv or None, B, Hq, Hkv, Nq, Nk, D, dtype, _strides_arg(strides), causal, window_left,
                        window_right, scale, workspace or None, workspace_bytes, stream or None)


def attn_bwd_workspace_size(B, Hq, Nq, D) -> int:
    return load_library().attn_bwd_workspace_size(B, Hq, Nq, D)


def attn_fwd_splitkv_noalloc(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, dtype, strides, causal, window_left,
                             window_right, scale, num_splits, stream):
    """C ``attn_fwd_splitkv_noalloc``: the split-KV call on the library's
    fixed 16 MiB scratch (no workspace argument)."""
    lib = load_library()
    return lib.attn_fwd_splitkv_noalloc(q or None, k or None, v or None, o or None, lse or None, B, Hq, Hkv, Nq, Nk,
                                        D, dtype, _strides_arg(strides), causal, window_left, window_right, scale,
                                        num_splits, stream or None)


def attn_fwd_splitkv_workspace_size(B, Hq, Nq, D, num_splits) -> int:
    return load_library().attn_fwd_splitkv_workspace_size(B, Hq, Nq, D, num_splits)


def attn_fwd_splitkv_plan(B, Hq, Hkv, Nq, Nk):
    """(status, num_splits) for the current device."""
    out = _int(0)
    rc = load_library().attn_fwd_splitkv_plan(B, Hq, Hkv, Nq, Nk, ctypes.byref(out))
    return rc, out.value


def attn_fwd_varlen_ex(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, cu_seqlens_q_host, cu_seqlens_k_host, num_seqs,
                       max_seqlen_q, max_seqlen_k, total_q, total_k, Hq, Hkv, D, dtype, strides, causal, window_left,
                       window_right, scale, stream):
    """C ``attn_fwd_varlen_ex``: pointers (device offsets and optional host
    mirrors) as ints; ``strides`` 12 ints."""
    lib = load_library()
    return lib.attn_fwd_varlen_ex(q or None, k or None, v or None, o or None, lse or None, cu_seqlens_q or None,
                                  cu_seqlens_k or None, cu_seqlens_q_host or None, cu_seqlens_k_host or None,
                                  num_seqs, max_seqlen_q, max_seqlen_k, total_q, total_k, Hq, Hkv, D, dtype,
                                  _strides_arg(strides), causal, window_left, window_right, scale, stream or None)


def attn_fwd_varlen(q, k, v, o, lse, cu_seqlens, cu_seqlens_host, num_seqs, max_seqlen, total_tokens, Hq, Hkv, D,
                    dtype, strides, causal, scale, stream):
    """C ``attn_fwd_varlen``: pointers as ints; ``cu_seqlens_host`` is an int
    address of a host int32 array or 0; ``strides`` 12 ints."""
    lib = load_library()
    return lib.attn_fwd_varlen(q or None, k or None, v or None, o or None, lse or None, cu_seqlens or None,
                               cu_seqlens_host or None, num_seqs, max_seqlen, total_tokens, Hq, Hkv, D, dtype,
                               _strides_arg(strides), causal, scale, stream or None)


def attn_fwd_host(q_host, k_host, v_host, o_host, lse_host, q_dev, k_dev, v_dev, o_dev, lse_dev, B, Hq, Hkv, N, D,
                  dtype, causal, scale, stream):
    """C ``attn_fwd_host``: host and device buffer addresses as ints."""
    lib = load_library()
    return lib.attn_fwd_host(q_host or None, k_host or None, v_host or None, o_host or None, lse_host or None,
                             q_dev or None, k_dev or None, v_dev or None, o_dev or None, lse_dev or None, B, Hq,
                             Hkv, N, D, dtype, causal, scale, stream or None)


def attn_fwd_varlen_host_plan(cu_seqlens, max_chunks=8):
    """C ``attn_fwd_varlen_host_plan`` on a host sequence of offsets: (status
    or chunk count k, the k + 1 run bounds)."""
    cu = (ctypes.c_int32 * max(len(cu_seqlens), 1))(*[int(x) for x in cu_seqlens])
    bounds = (ctypes.c_int32 * 9)()
    k = load_library().attn_fwd_varlen_host_plan(ctypes.addressof(cu), len(cu_seqlens) - 1, max_chunks, bounds)
    return k, list(bounds[:k + 1]) if k > 0 else []


def attn_fwd_varlen_host(q_host, k_host, v_host, o_host, lse_host, cu_seqlens_host, q_dev, k_dev, v_dev, o_dev,
                         lse_dev, cu_seqlens_dev, num_seqs, max_seqlen, total_tokens, Hq, Hkv, D, dtype, causal,
                         scale, stream):
    """C ``attn_fwd_varlen_host``: host and device buffer addresses as ints."""
    lib = load_library()
    return lib.attn_fwd_varlen_host(q_host or None, k_host or None, v_host or None, o_host or None,
                                    lse_host or None, cu_seqlens_host or None, q_dev or None, k_dev or None,
                                    v_dev or None, o_dev or None, lse_dev or None, cu_seqlens_dev or None,
                                    num_seqs, max_seqlen, total_tokens, Hq, Hkv, D, dtype, causal, scale,
                                    stream or None)


def attn_qk_norm_rope(q, k, q_weight, k_weight, rope_cos, rope_sin, positions, q_out, k_out, total_tokens, Hq, Hk, D,
                      dtype, strides, rope_dim, interleaved, max_position, eps, stream):
    """C ``attn_qk_norm_rope``: pointers as ints (0 for NULL), ``strides`` 12 ints."""
    lib = load_library()
    return lib.attn_qk_norm_rope(q or None, k or None, q_weight or None, k_weight or None, rope_cos or None,
                                 rope_sin or None, positions or None, q_out or None, k_out or None, total_tokens, Hq,
                                 Hk, D, dtype, _STRIDES[12](*strides), rope_dim, interleaved, max_position, eps,
                                 stream or None)


def attn_qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight, k_weight, rope_cos, rope_sin, positions, dq, dk, dq_weight,
                          dk_weight, total_tokens, Hq, Hk, D, dtype, strides, rope_dim, interleaved, max_position,
                          eps, workspace, workspace_bytes, stream):
    """C ``attn_qk_norm_rope_bwd``: pointers as ints (0 for NULL), ``strides`` 18 ints."""
    lib = load_library()
    return lib.attn_qk_norm_rope_bwd(q or None, k or None, dq_out or None, dk_out or None, q_weight or None,
                                     k_weight or None, rope_cos or None, rope_sin or None, positions or None,
                                     dq or None, dk or None, dq_weight or None, dk_weight or None, total_tokens, Hq,
                                     Hk, D, dtype, _STRIDES[18](*strides), rope_dim, interleaved, max_position, eps,
                                     workspace or None, workspace_bytes, stream or None)


def attn_qk_norm_rope_bwd_workspace_size(total_tokens, Hq, Hk, D) -> int:
    return load_library().attn_qk_norm_rope_bwd_workspace_size(total_tokens, Hq, Hk, D)


def attn_paged_append(q, k, v, q_weight, k_weight, rope_cos, rope_sin, q_out, k_pages, v_pages, block_table, seqlens_k,
                      cu_seqlens_q, num_seqs, total_tokens, Hq, Hkv, D, dtype, strides, page_size, num_pages,
                      max_pages, table_stride, rope_dim, interleaved, max_position, eps, stream):
    """C ``attn_paged_append``: pointers as ints (0 for NULL), ``strides`` 20 ints."""
    lib = load_library()
    return lib.attn_paged_append(q or None, k or None, v or None, q_weight or None, k_weight or None,
                                 rope_cos or None, rope_sin or None, q_out or None, k_pages or None, v_pages or None,
                                 block_table or None, seqlens_k or None, cu_seqlens_q or None, num_seqs, total_tokens,
                                 Hq, Hkv, D, dtype, _STRIDES[20](*strides), page_size, num_pages, max_pages,
                                 table_stride, rope_dim, interleaved, max_position, eps, stream or None)


def attn_fwd_paged(q, k_pages, v_pages, o, lse, block_table, seqlens_k, cu_seqlens_q, num_seqs, max_seqlen_q, total_q,
                   Hq, Hkv, D, dtype, strides, page_size, num_pages, max_pages, table_stride, causal, window_left,
                   window_right, scale, num_shares, workspace, workspace_bytes, stream):
    """C ``attn_fwd_paged``: pointers as ints (0 for NULL), ``strides`` 14 ints."""
    lib = load_library()
    return lib.attn_fwd_paged(q or None, k_pages or None, v_pages or None, o or None, lse or None, block_table or None,
                              seqlens_k or None, cu_seqlens_q or None, num_seqs, max_seqlen_q, total_q, Hq, Hkv, D,
                              dtype, _STRIDES[14](*strides), page_size, num_pages, max_pages, table_stride, causal,
                              window_left, window_right, scale, num_shares, workspace or None, workspace_bytes,
                              stream or None)


def attn_fwd_paged_workspace_size(Hq, Hkv, max_seqlen_q, D, num_shares) -> int:
    return load_library().attn_fwd_paged_workspace_size(Hq, Hkv, max_seqlen_q, D, num_shares)


def attn_fwd_paged_plan(num_seqs, Hq, Hkv, max_seqlen_q, max_seqlen_k, D, num_shares=0):
    """(status, num_shares, workspace bytes) for the current device."""
    shares, need = _int(num_shares), ctypes.c_size_t(0)
    rc = load_library().attn_fwd_paged_plan(num_seqs, Hq, Hkv, max_seqlen_q, max_seqlen_k, D, ctypes.byref(shares),
                                            ctypes.byref(need))
    return rc, shares.value, need.value


def etattn_status_string(code: int) -> str:
    return load_library().etattn_status_string(code).decode()


def etattn_last_cuda_error() -> int:
    return load_library().etattn_last_cuda_error()


def etattn_read_device_status(clear: bool = True, stream: int = 0) -> int:
    out = _int(0)
    rc = load_library().etattn_read_device_status(ctypes.byref(out), 1 if clear else 0, stream or None)
    if rc != 0:
        raise EtattnError(rc, "etattn_read_device_status")
    return out.value


def etattn_version() -> int:
    return load_library().etattn_version()


def etattn_selftest_wait_timeout(limit_us: int, stream: int = 0) -> int:
    """C ``etattn_selftest_wait_timeout``: enqueue the bounded-wait self-test
    (a wait of limit_us microseconds that runs out and sets the device status
    word).  Returns the status code."""
    return load_library().etattn_selftest_wait_timeout(limit_us, stream or None)


# ---------------------------------------------------------------- torch marshalling

def _dtype_code(t):
    import torch
    if t.dtype == torch.float16:
        return ETATTN_F16
    if t.dtype == torch.bfloat16:
        return ETATTN_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; expected float16 or bfloat16")


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def attention(q, k, v, *, causal: bool = True, scale: float | None = None, window_left: int = -1,
              window_right: int = -1, out=None, lse=None, return_lse: bool = True, stream=None):
    """Batched (GQA-capable) attention on CUDA tensors.

    q: [B, Hq, Nq, D]; k, v: [B, Hkv, Nk, D] (any strides with d contiguous,
    e.g. a [B, N, H, D] buffer viewed through permute).  With Nk != Nq the
    last query row aligns with the last key; ``window_left`` /
    ``window_right`` >= 0 bound the keys a row reads around its own key
    position.  Returns (o, lse) with o a new [B, Hq, Nq, D] tensor (or
    ``out``) and lse a new [B, Hq, Nq] FP32 tensor (or ``lse``; None when
    ``return_lse`` is False).  Square calls without a window go through
    ``attn_fwd``, the others through ``attn_fwd_ex``."""
    import torch
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((B, Hq, Nq, D), dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, Nq) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [B, Hq, Nq] tensor")
    strides = [*q.stride(), *k.stride(), *v.stride(), *out.stride()]
    lse_ptr = lse.data_ptr() if lse is not None else 0
    square = Nq == Nk and window_left < 0 and window_right < 0
    with torch.cuda.device(q.device):
        if square:
            rc = attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr, B, Hq, Hkv, Nq, D,
                          _dtype_code(q), strides, 1 if causal else 0, float(scale), _stream_handle(stream))
        else:
            rc = attn_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr, B, Hq, Hkv, Nq, Nk,
                             D, _dtype_code(q), strides, 1 if causal else 0, int(window_left), int(window_right),
                             float(scale), _stream_handle(stream))
    if rc != 0:
        raise EtattnError(rc, "attn_fwd" if square else "attn_fwd_ex")
    return out, lse


def attention_splitkv(q, k, v, *, causal: bool = True, scale: float | None = None, window_left: int = -1,
                      window_right: int = -1, num_splits: int | None = None, workspace=None, out=None, lse=None,
                      return_lse: bool = True, stream=None):
    """``attention`` computed with the keys cut into ``num_splits`` slices
    (default: the library's plan for the current device) and merged by a
    second launch.  ``workspace`` is a CUDA uint8 tensor of at least
    ``attn_fwd_splitkv_workspace_size`` bytes (allocated here when None)."""
    import torch
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(q.device):
        if num_splits is None:
            rc, num_splits = attn_fwd_splitkv_plan(B, Hq, Hkv, Nq, Nk)
            if rc != 0:
                raise EtattnError(rc, "attn_fwd_splitkv_plan")
        need = attn_fwd_splitkv_workspace_size(B, Hq, Nq, D, num_splits)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        if out is None:
            out = torch.empty((B, Hq, Nq, D), dtype=q.dtype, device=q.device)
        if lse is None and return_lse:
            lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
        strides = [*q.stride(), *k.stride(), *v.stride(), *out.stride()]
        ws_ptr = workspace.data_ptr() if workspace is not None else 0
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        rc = attn_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                              lse.data_ptr() if lse is not None else 0, B, Hq, Hkv, Nq, Nk, D, _dtype_code(q),
                              strides, 1 if causal else 0, int(window_left), int(window_right), float(scale),
                              int(num_splits), ws_ptr, ws_bytes, _stream_handle(stream))
    if rc != 0:
        raise EtattnError(rc, "attn_fwd_splitkv")
    return out, lse


def attention_global(q, k, v, *, num_global: int, causal: bool = True, scale: float | None = None,
                     window_left: int = -1, window_right: int = -1, out=None, lse=None, return_lse: bool = True,
                     stream=None):
    """``attention`` with ``num_global`` global tokens beside the window (the
    first positions read and are read by every row, under the causal mask)."""
    import torch
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(q.device):
        if out is None:
            out = torch.empty((B, Hq, Nq, D), dtype=q.dtype, device=q.device)
        if lse is None and return_lse:
            lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
        strides = [*q.stride(), *k.stride(), *v.stride(), *out.stride()]
        rc = attn_fwd_global(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                             lse.data_ptr() if lse is not None else 0, B, Hq, Hkv, Nq, Nk, D, _dtype_code(q), strides,
                             1 if causal else 0, int(window_left), int(window_right), int(num_global), float(scale),
                             _stream_handle(stream))
    if rc != 0:
        raise EtattnError(rc, "attn_fwd_global")
    return out, lse


def attention_backward(q, k, v, o, lse, dout, *, causal: bool = True, scale: float | None = None,
                       window_left: int = -1, window_right: int = -1, dq=None, dk=None, dv=None, workspace=None,
                       stream=None):
    """Gradients (dq, dk, dv) of ``attention`` for upstream gradient ``dout``,
    given the forward's output ``o`` and logsumexp ``lse`` ([B, Hq, Nq] FP32).
    Shapes and strides as for ``attention``; the outputs are allocated when
    not given, and so is the FP32 workspace (``attn_bwd_workspace_size``)."""
    import torch
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, Nq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, Hq, Nq] tensor")
    with torch.cuda.device(q.device):
        if dq is None:
            dq = torch.empty((B, Hq, Nq, D), dtype=q.dtype, device=q.device)
        if dk is None:
            dk = torch.empty((B, Hkv, Nk, D), dtype=q.dtype, device=q.device)
        if dv is None:
            dv = torch.empty((B, Hkv, Nk, D), dtype=q.dtype, device=q.device)
        need = attn_bwd_workspace_size(B, Hq, Nq, D)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        strides = [*q.stride(), *k.stride(), *v.stride(), *o.stride(), *dout.stride(), *dq.stride(), *dk.stride(),
                   *dv.stride()]
        ws_ptr = workspace.data_ptr() if workspace is not None else 0
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        rc = attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                      dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Nq, Nk, D, _dtype_code(q), strides,
                      1 if causal else 0, int(window_left), int(window_right), float(scale), ws_ptr, ws_bytes,
                      _stream_handle(stream))
    if rc != 0:
        raise EtattnError(rc, "attn_bwd")
    return dq, dk, dv


def attn_fwd_varlen_splitkv(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, cu_seqlens_q_host, cu_seqlens_k_host,
                            num_seqs, max_seqlen_q, max_seqlen_k, total_q, total_k, Hq, Hkv, D, dtype, strides, causal,
                            window_left, window_right, scale, num_splits, workspace, workspace_bytes, stream):
    """C ``attn_fwd_varlen_splitkv``: pointers as ints; ``strides`` 12 ints."""
    lib = load_library()
    return lib.attn_fwd_varlen_splitkv(q or None, k or None, v or None, o or None, lse or None, cu_seqlens_q or None,
                                       cu_seqlens_k or None, cu_seqlens_q_host or None, cu_seqlens_k_host or None,
                                       num_seqs, max_seqlen_q, max_seqlen_k, total_q, total_k, Hq, Hkv, D, dtype,
                                       _strides_arg(strides), causal, window_left, window_right, scale, num_splits,
                                       workspace or None, workspace_bytes, stream or None)


def attn_fwd_varlen_splitkv_plan(num_seqs, Hq, Hkv, max_seqlen_q, max_seqlen_k):
    """(status, num_splits) for the current device."""
    out = _int(0)
    rc = load_library().attn_fwd_varlen_splitkv_plan(num_seqs, Hq, Hkv, max_seqlen_q, max_seqlen_k,
                                                      ctypes.byref(out))
    return rc, out.value


def attn_fwd_varlen_splitkv_workspace_size(total_q, Hq, D, num_splits) -> int:
    return load_library().attn_fwd_varlen_splitkv_workspace_size(total_q, Hq, D, num_splits)


def attn_fwd_varlen_global(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, cu_seqlens_q_host, cu_seqlens_k_host,
                           num_seqs, max_seqlen_q, max_seqlen_k, total_q, total_k, Hq, Hkv, D, dtype, strides, causal,
                           window_left, window_right, num_global, scale, stream):
    """C ``attn_fwd_varlen_global``: pointers as ints; ``strides`` 12 ints."""
    lib = load_library()
    return lib.attn_fwd_varlen_global(q or None, k or None, v or None, o or None, lse or None, cu_seqlens_q or None,
                                      cu_seqlens_k or None, cu_seqlens_q_host or None, cu_seqlens_k_host or None,
                                      num_seqs, max_seqlen_q, max_seqlen_k, total_q, total_k, Hq, Hkv, D, dtype,
                                      _strides_arg(strides), causal, window_left, window_right, num_global, scale,
                                      stream or None)


def attention_varlen(q, k, v, cu_seqlens, max_seqlen: int, *, causal: bool = True, scale: float | None = None,
                     cu_seqlens_k=None, max_seqlen_k: int | None = None, window_left: int = -1,
                     window_right: int = -1, cu_seqlens_host=None, cu_seqlens_k_host=None, out=None, lse=None,
                     return_lse: bool = True, stream=None, num_splits: int = 1, num_global: int = 0,
                     workspace=None):
    """Packed variable-length attention on CUDA tensors.

    q: [T, Hq, D]; k, v: [Tk, Hkv, D]; cu_seqlens: int32 CUDA tensor [S+1]
    of query offsets; ``cu_seqlens_k`` (default: cu_seqlens) the key
    offsets, with ``max_seqlen_k`` their longest length.  The host mirrors
    ``cu_seqlens_host`` / ``cu_seqlens_k_host`` (optional int32 CPU tensors)
    are validated before launch.  Returns (o [T, Hq, D], lse [Hq, T] FP32 or
    None).  Self-attention without a window goes through
    ``attn_fwd_varlen``, the rest through ``attn_fwd_varlen_ex``; with
    ``num_splits`` > 1 through ``attn_fwd_varlen_splitkv`` and with
    ``num_global`` > 0 through ``attn_fwd_varlen_global`` (``workspace``: the
    split-KV scratch, a CUDA uint8 tensor allocated here when None)."""
    import torch
    T, Hq, D = q.shape
    Tk, Hkv = k.shape[0], k.shape[1]
    S = cu_seqlens.shape[0] - 1
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    for name, t in (("cu_seqlens", cu_seqlens), ("cu_seqlens_k", cu_seqlens_k)):
        if t is not None and (t.dtype != torch.int32 or not t.is_cuda):
            raise TypeError(f"{name} must be an int32 CUDA tensor")
    if out is None:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)

    def host_addr(t):
        if t is None:
            return None, 0
        t = t.to(torch.int32).contiguous()
        return t, t.data_ptr()

    cu_host, host_ptr = host_addr(cu_seqlens_host)
    cu_k_host, host_k_ptr = host_addr(cu_seqlens_k_host)
    strides = [*q.stride(), *k.stride(), *v.stride(), *out.stride()]
    lse_ptr = lse.data_ptr() if lse is not None else 0
    plain = (cu_seqlens_k is None and cu_k_host is None and window_left < 0 and window_right < 0 and num_splits <= 1
             and num_global <= 0)
    with torch.cuda.device(q.device):
        if num_global > 0 or num_splits > 1:
            cu_k = cu_seqlens if cu_seqlens_k is None else cu_seqlens_k
            if cu_seqlens_k is None:
                host_k_ptr = host_ptr
            mk = int(max_seqlen if max_seqlen_k is None else max_seqlen_k)
            need = 0 if num_global > 0 else attn_fwd_varlen_splitkv_workspace_size(T, Hq, D, int(num_splits))
            if workspace is None and need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            ws_ptr = workspace.data_ptr() if workspace is not None else 0
            ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
            common = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr, cu_seqlens.data_ptr(),
                      cu_k.data_ptr(), host_ptr, host_k_ptr, S, int(max_seqlen), mk, T, Tk, Hq, Hkv, D,
                      _dtype_code(q), strides, 1 if causal else 0, int(window_left), int(window_right))
            if num_global > 0:
                rc = attn_fwd_varlen_global(*common, int(num_global), float(scale), _stream_handle(stream))
                name = "attn_fwd_varlen_global"
            else:
                rc = attn_fwd_varlen_splitkv(*common, float(scale), int(num_splits), ws_ptr, ws_bytes,
                                             _stream_handle(stream))
                name = "attn_fwd_varlen_splitkv"
        elif plain:
            rc = attn_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr,
                                 cu_seqlens.data_ptr(), host_ptr, S, int(max_seqlen), T, Hq, Hkv, D, _dtype_code(q),
                                 strides, 1 if causal else 0, float(scale), _stream_handle(stream))
        else:
            cu_k = cu_seqlens if cu_seqlens_k is None else cu_seqlens_k
            if cu_seqlens_k is None:
                host_k_ptr = host_ptr
            mk = int(max_seqlen if max_seqlen_k is None else max_seqlen_k)
            rc = attn_fwd_varlen_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr,
                                    cu_seqlens.data_ptr(), cu_k.data_ptr(), host_ptr, host_k_ptr, S, int(max_seqlen),
                                    mk, T, Tk, Hq, Hkv, D, _dtype_code(q), strides, 1 if causal else 0,
                                    int(window_left), int(window_right), float(scale), _stream_handle(stream))
    del cu_host, cu_k_host
    if rc != 0:
        if num_global <= 0 and num_splits <= 1:
            name = "attn_fwd_varlen" if plain else "attn_fwd_varlen_ex"
        raise EtattnError(rc, name)
    return out, lse


# The calls of one decode step take a few microseconds on the device, so the
# helpers below keep their own time down: one comparison per tensor on the way
# through (the messages are made when it fails), strides packed into bytes, the
# device made current (by a second call of the helper) only when it is not, and
# the C functions called directly.  (``empty_like`` and ``empty`` with its sizes
# as arguments take half the time of ``empty`` with a tuple.)

_STRIDES = {n: struct.Struct(f"{n}q").pack for n in (12, 14, 18, 20)}
_CODES: dict = {}  # torch dtype -> ETATTN_* code


@functools.lru_cache(maxsize=512)
def _paged_plan(device_index, num_seqs, Hq, Hkv, max_seqlen_q, max_seqlen_k, D, num_shares):
    """attn_fwd_paged_plan on the current device (``device_index``): a function of the sizes alone."""
    rc, shares, need = attn_fwd_paged_plan(num_seqs, Hq, Hkv, max_seqlen_q, max_seqlen_k, D, num_shares)
    if rc != 0:
        raise EtattnError(rc, "attn_fwd_paged_plan")
    return shares, need


@functools.lru_cache(maxsize=512)
def _rope_bwd_bytes(T, Hq, Hk, D):
    return attn_qk_norm_rope_bwd_workspace_size(T, Hq, Hk, D)


def _code_of(t):
    """The element type's code; a TypeError for another type."""
    code = _CODES.get(t.dtype)
    if code is None:
        code = _CODES[t.dtype] = _dtype_code(t)
    return code


def _elsewhere(torch, device, stream):
    """The context in which a helper has to call itself again, so that what it
    allocates and launches belongs to ``stream`` and ``device``; None when it
    is there already.  A ValueError for tensors or a stream of another kind."""
    if device.type != "cuda":
        raise ValueError(f"expected CUDA tensors, got tensors on {device}")
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    return None if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _check(name, t, shape, dtype, device, dense=False):
    """Raises for a tensor argument that is not as it must be."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rope_args(torch, D, dtype, device, q_weight, k_weight, rope_cos, rope_sin):
    """(addresses of the weights and tables, rope_dim, max_position), after checking them."""
    wq = wk = cos = sin = rope_dim = max_position = 0
    if q_weight is not None:
        if q_weight.shape != (D,) or q_weight.dtype != dtype or q_weight.device != device or not q_weight.is_contiguous():
            _check("q_weight", q_weight, (D,), dtype, device, True)
        wq = q_weight.data_ptr()
    if k_weight is not None:
        if k_weight.shape != (D,) or k_weight.dtype != dtype or k_weight.device != device or not k_weight.is_contiguous():
            _check("k_weight", k_weight, (D,), dtype, device, True)
        wk = k_weight.data_ptr()
    if rope_cos is not None and rope_sin is not None:
        shape = rope_cos.shape
        if len(shape) != 2:
            raise ValueError("rope_cos and rope_sin must be [max_position, rope_dim / 2]")
        if (rope_cos.dtype != torch.float32 or rope_cos.device != device or not rope_cos.is_contiguous()
                or rope_sin.shape != shape or rope_sin.dtype != torch.float32 or rope_sin.device != device
                or not rope_sin.is_contiguous()):
            _check("rope_cos", rope_cos, shape, torch.float32, device, True)
            _check("rope_sin", rope_sin, shape, torch.float32, device, True)
        max_position, rope_dim = shape
        rope_dim *= 2
        cos, sin = rope_cos.data_ptr(), rope_sin.data_ptr()
    elif rope_cos is not rope_sin:
        raise ValueError("rope_cos and rope_sin come together")
    return wq, wk, cos, sin, rope_dim, max_position


def _positions(torch, positions, T, rope_dim, device):
    """The address of the tokens' positions, after checking them."""
    if positions is None:
        if rope_dim:
            raise ValueError("positions are needed with rope_cos and rope_sin")
        return 0
    if (positions.shape != (T,) or positions.dtype != torch.int32 or positions.device != device
            or not positions.is_contiguous()):
        _check("positions", positions, (T,), torch.int32, device, True)
    return positions.data_ptr()


def rope_tables(max_position: int, rope_dim: int, *, theta: float = 10000.0, device=None):
    """(rope_cos, rope_sin): FP32 [max_position, rope_dim / 2] tables of the angles
    position * theta^(-2i / rope_dim), from angles in 64 bits (an angle of a far
    position has no correct digit left in 32)."""
    import torch
    device = torch.device("cuda") if device is None else device
    inv = theta ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=device) / rope_dim)
    angle = torch.arange(max_position, dtype=torch.float64, device=device)[:, None] * inv
    return angle.cos().float(), angle.sin().float()


def qk_norm_rope(q, k, *, q_weight=None, k_weight=None, rope_cos=None, rope_sin=None, positions=None,
                 interleaved: bool = False, eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """RMS norm of every head and rotation by position of q [T, Hq, D] and k
    [T, Hk, D] in one pass; returns (q_out, k_out), new tensors when not given.

    ``q_weight`` / ``k_weight`` ([D], q's dtype): the norm's weights, None for
    no norm.  ``rope_cos`` / ``rope_sin`` (FP32 [max_position, rope_dim / 2],
    see ``rope_tables``) and ``positions`` (int32 [T]): the rotation, None for
    none.  Views of a fused projection serve as q and k."""
    import torch
    T, Hq, D = q.shape
    Hk, dtype, device, code = k.shape[1], q.dtype, q.device, _code_of(q)
    if k.shape != (T, Hk, D) or k.dtype != dtype or k.device != device:
        _check("k", k, (T, Hk, D), dtype, device)
    wq, wk, cos, sin, rope_dim, max_position = _rope_args(torch, D, dtype, device, q_weight, k_weight, rope_cos,
                                                          rope_sin)
    pos = _positions(torch, positions, T, rope_dim, device)
    if q_out is not None:
        _check("q_out", q_out, (T, Hq, D), dtype, device)
    if k_out is not None:
        _check("k_out", k_out, (T, Hk, D), dtype, device)
    there = _elsewhere(torch, device, stream)
    if there is not None:
        with there:
            return qk_norm_rope(q, k, q_weight=q_weight, k_weight=k_weight, rope_cos=rope_cos, rope_sin=rope_sin,
                                positions=positions, interleaved=interleaved, eps=eps, q_out=q_out, k_out=k_out)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if k_out is None:
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
    rc = (_lib or load_library()).attn_qk_norm_rope(
        q.data_ptr(), k.data_ptr(), wq, wk, cos, sin, pos, q_out.data_ptr(), k_out.data_ptr(), T, Hq, Hk, D, code,
        _STRIDES[12](*q.stride(), *k.stride(), *q_out.stride(), *k_out.stride()), rope_dim, interleaved,
        max_position, eps, torch._C._cuda_getCurrentRawStream(device.index))
    if rc != 0:
        raise EtattnError(rc, "attn_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(q, k, dq_out, dk_out, *, q_weight=None, k_weight=None, rope_cos=None, rope_sin=None,
                          positions=None, interleaved: bool = False, eps: float = 1e-6, dq=None, dk=None,
                          workspace=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of ``qk_norm_rope`` for the
    upstream gradients ``dq_out`` and ``dk_out`` (not broadcast ones: a stride of
    0 is refused); the weights' are FP32 [D] (None without the weight)."""
    import torch
    T, Hq, D = q.shape
    Hk, dtype, device, code = k.shape[1], q.dtype, q.device, _code_of(q)
    if (k.shape != (T, Hk, D) or k.dtype != dtype or k.device != device or dq_out.shape != q.shape
            or dq_out.dtype != dtype or dq_out.device != device or dk_out.shape != k.shape or dk_out.dtype != dtype
            or dk_out.device != device):
        _check("k", k, (T, Hk, D), dtype, device)
        _check("dq_out", dq_out, (T, Hq, D), dtype, device)
        _check("dk_out", dk_out, (T, Hk, D), dtype, device)
    wq, wk, cos, sin, rope_dim, max_position = _rope_args(torch, D, dtype, device, q_weight, k_weight, rope_cos,
                                                          rope_sin)
    pos = _positions(torch, positions, T, rope_dim, device)
    if dq is not None:
        _check("dq", dq, (T, Hq, D), dtype, device)
    if dk is not None:
        _check("dk", dk, (T, Hk, D), dtype, device)
    there = _elsewhere(torch, device, stream)
    if there is not None:
        with there:
            return qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight=q_weight, k_weight=k_weight,
                                         rope_cos=rope_cos, rope_sin=rope_sin, positions=positions,
                                         interleaved=interleaved, eps=eps, dq=dq, dk=dk, workspace=workspace)
    lib = _lib or load_library()
    if dq is None:
        dq = torch.empty_like(q, memory_format=torch.contiguous_format)
    if dk is None:
        dk = torch.empty_like(k, memory_format=torch.contiguous_format)
    dwq = torch.empty(D, dtype=torch.float32, device=device) if wq else None
    dwk = torch.empty(D, dtype=torch.float32, device=device) if wk else None
    ws_bytes = 0
    if workspace is not None:
        ws_bytes = _workspace(workspace, device)
    elif wq or wk:
        ws_bytes = _rope_bwd_bytes(T, Hq, Hk, D)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
    rc = lib.attn_qk_norm_rope_bwd(
        q.data_ptr(), k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(), wq, wk, cos, sin, pos, dq.data_ptr(),
        dk.data_ptr(), dwq.data_ptr() if wq else 0, dwk.data_ptr() if wk else 0, T, Hq, Hk, D, code,
        _STRIDES[18](*q.stride(), *k.stride(), *dq_out.stride(), *dk_out.stride(), *dq.stride(), *dk.stride()),
        rope_dim, interleaved, max_position, eps, workspace.data_ptr() if ws_bytes else 0, ws_bytes,
        torch._C._cuda_getCurrentRawStream(device.index))
    if rc != 0:
        raise EtattnError(rc, "attn_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


def _workspace(t, device):
    """The bytes of a given workspace."""
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return t.numel() * t.element_size()


def _page_args(torch, k_pages, v_pages, block_table, seqlens_k, cu_seqlens_q, dtype, device):
    """(num_seqs, max_pages, table_stride, address of the offsets), after checking the cache's tensors."""
    shape = k_pages.shape
    if len(shape) != 4:
        raise ValueError("k_pages must be [num_pages, Hkv, page_size, D]")
    S, width = block_table.shape
    row, col = block_table.stride()
    if (k_pages.dtype != dtype or k_pages.device != device or v_pages.shape != shape or v_pages.dtype != dtype
            or v_pages.device != device or block_table.dtype != torch.int32 or block_table.device != device
            or seqlens_k.shape != (S,) or seqlens_k.dtype != torch.int32 or seqlens_k.device != device
            or not seqlens_k.is_contiguous()):
        _check("k_pages", k_pages, shape, dtype, device)
        _check("v_pages", v_pages, shape, dtype, device)
        _check("block_table", block_table, (S, width), torch.int32, device)
        _check("seqlens_k", seqlens_k, (S,), torch.int32, device, True)
    if col != 1 and width > 1:
        raise ValueError("block_table's rows must be contiguous")
    if cu_seqlens_q is None:
        return S, width, row, 0
    _check("cu_seqlens_q", cu_seqlens_q, (S + 1,), torch.int32, device, True)
    return S, width, row, cu_seqlens_q.data_ptr()


def paged_append(k, v, k_pages, v_pages, block_table, seqlens_k, *, q=None, q_weight=None, k_weight=None,
                 rope_cos=None, rope_sin=None, interleaved: bool = False, eps: float = 1e-6, cu_seqlens_q=None,
                 q_out=None, stream=None):
    """Writes this step's keys and values k, v [T, Hkv, D] into the paged cache,
    the keys normed and rotated at their positions on the way (as
    ``qk_norm_rope``), and returns q [T, Hq, D] normed and rotated (None
    without q).

    k_pages, v_pages: logical [num_pages, Hkv, page_size, D] (any strides with d
    contiguous); block_table: int32 [S, max_pages]; seqlens_k: int32 [S], the
    keys of every sequence with the new ones; cu_seqlens_q: int32 [S + 1]
    offsets of the new tokens, None when every sequence has T / S."""
    import torch
    T, _, D = k.shape
    dtype, device, code = k.dtype, k.device, _code_of(k)
    S, width, row, cu = _page_args(torch, k_pages, v_pages, block_table, seqlens_k, cu_seqlens_q, dtype, device)
    num_pages, Hkv, page_size, Dp = k_pages.shape
    if k.shape != (T, Hkv, Dp) or v.shape != (T, Hkv, Dp) or v.dtype != dtype or v.device != device:
        _check("k", k, (T, Hkv, Dp), dtype, device)
        _check("v", v, (T, Hkv, Dp), dtype, device)
    wq, wk, cos, sin, rope_dim, max_position = _rope_args(torch, D, dtype, device, q_weight, k_weight, rope_cos,
                                                          rope_sin)
    Hq = 0
    if q is not None:
        Hq = q.shape[1]
        if q.shape != (T, Hq, D) or q.dtype != dtype or q.device != device:
            _check("q", q, (T, Hq, D), dtype, device)
        if q_out is not None:
            _check("q_out", q_out, (T, Hq, D), dtype, device)
    there = _elsewhere(torch, device, stream)
    if there is not None:
        with there:
            return paged_append(k, v, k_pages, v_pages, block_table, seqlens_k, q=q, q_weight=q_weight,
                                k_weight=k_weight, rope_cos=rope_cos, rope_sin=rope_sin, interleaved=interleaved,
                                eps=eps, cu_seqlens_q=cu_seqlens_q, q_out=q_out)
    if q is None:
        q_out, qp, op, q_stride, o_stride = None, 0, 0, (0, 0, 1), (0, 0, 1)
    else:
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        qp, op, q_stride, o_stride = q.data_ptr(), q_out.data_ptr(), q.stride(), q_out.stride()
    rc = (_lib or load_library()).attn_paged_append(
        qp, k.data_ptr(), v.data_ptr(), wq, wk, cos, sin, op, k_pages.data_ptr(), v_pages.data_ptr(),
        block_table.data_ptr(), seqlens_k.data_ptr(), cu, S, T, Hq, Hkv, D, code,
        _STRIDES[20](*q_stride, *k.stride(), *v.stride(), *o_stride, *k_pages.stride(), *v_pages.stride()),
        page_size, num_pages, width, row, rope_dim, interleaved, max_position, eps,
        torch._C._cuda_getCurrentRawStream(device.index))
    if rc != 0:
        raise EtattnError(rc, "attn_paged_append")
    return q_out


def attention_paged(q, k_pages, v_pages, block_table, seqlens_k, *, cu_seqlens_q=None, max_seqlen_q: int | None = None,
                    max_seqlen_k: int | None = None, causal: bool = True, scale: float | None = None,
                    window_left: int = -1, window_right: int = -1, num_shares: int | None = None, workspace=None,
                    out=None, lse=None, return_lse: bool = True, stream=None):
    """Attention of the new tokens q [T, Hq, D] over a paged cache; returns
    (o [T, Hq, D], lse [Hq, T] FP32 or None).

    k_pages, v_pages, block_table, seqlens_k, cu_seqlens_q: as for
    ``paged_append``; with cu_seqlens_q, ``max_seqlen_q`` (the most new tokens
    of a sequence) is needed too.  ``max_seqlen_k`` (default: what the block
    table can hold) only bounds the number of shares the work is cut into;
    ``num_shares`` (default: the library's plan for the current device) and
    ``workspace`` (a CUDA uint8 tensor of ``attn_fwd_paged_workspace_size``
    bytes) may be given, as a captured graph's owner would."""
    import torch
    T, Hq, D = q.shape
    dtype, device, code = q.dtype, q.device, _code_of(q)
    S, width, row, cu = _page_args(torch, k_pages, v_pages, block_table, seqlens_k, cu_seqlens_q, dtype, device)
    num_pages, Hkv, page_size, Dp = k_pages.shape
    if Dp != D:
        raise ValueError(f"k_pages has head dim {Dp}, q has {D}")
    if not cu:
        max_seqlen_q = T // S if S > 0 else 0
    elif max_seqlen_q is None:
        raise ValueError("max_seqlen_q is needed with cu_seqlens_q")
    if out is not None:
        _check("out", out, (T, Hq, D), dtype, device)
    if lse is not None:
        _check("lse", lse, (Hq, T), torch.float32, device, True)
    there = _elsewhere(torch, device, stream)
    if there is not None:
        with there:
            return attention_paged(q, k_pages, v_pages, block_table, seqlens_k, cu_seqlens_q=cu_seqlens_q,
                                   max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k, causal=causal, scale=scale,
                                   window_left=window_left, window_right=window_right, num_shares=num_shares,
                                   workspace=workspace, out=out, lse=lse, return_lse=return_lse)
    lib = _lib or load_library()
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None and return_lse:
        lse = torch.empty(Hq, T, dtype=torch.float32, device=device)
    if num_shares is None or workspace is None:
        if max_seqlen_k is None:
            max_seqlen_k = min(width * page_size, 1 << 30)
        num_shares, ws_bytes = _paged_plan(device.index, S, Hq, Hkv, int(max_seqlen_q), int(max_seqlen_k), D,
                                           int(num_shares or 0))
    if workspace is not None:
        ws_bytes = _workspace(workspace, device)
    elif ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
    rc = lib.attn_fwd_paged(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(),
        block_table.data_ptr(), seqlens_k.data_ptr(), cu, S, max_seqlen_q, T, Hq, Hkv, D, code,
        _STRIDES[14](*q.stride(), *k_pages.stride(), *v_pages.stride(), *out.stride()), page_size, num_pages, width,
        row, causal, window_left, window_right, D ** -0.5 if scale is None else scale, num_shares,
        0 if workspace is None else workspace.data_ptr(), ws_bytes, torch._C._cuda_getCurrentRawStream(device.index))
    if rc != 0:
        raise EtattnError(rc, "attn_fwd_paged")
    return out, lse
