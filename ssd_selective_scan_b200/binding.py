"""ctypes binding of libssd.so -- the C ABI declared in include/ssd.h and
include/ssd_diag.h.

Argument marshalling only: every function here passes integers (device
pointers, sizes, a cudaStream_t handle) straight to the C entry point of the
same name and returns its status code.  There is no computation and no
fallback: if libssd.so is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import sysconfig
import threading

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libssd.so")
PYCALL_PATH = os.path.join(PKG_DIR, "_pycall.so")

# ssd_status_t
SSD_OK = 0
SSD_ERR_INVALID_ARG = 1
SSD_ERR_UNSUPPORTED = 2
SSD_ERR_CUDA = 3
SSD_ERR_TIMEOUT = 4
# ssd_dtype_t
SSD_F32 = 0
SSD_BF16 = 1

# Every exported entry point and its ctypes signature (restype, argtypes).
_vp, _i, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "ssd_status_string": (ctypes.c_char_p, [_i]),
    "ssd_abi_version": (_i, []),
    "ssd_conv1d_silu": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "ssd_chunk_scan_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "ssd_chunk_scan_fwd": (_i, [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                _i, _i, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp, _vp]),
    "ssd_state_update": (_i, [_vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                              _i, _i, _i, _i, _i, _i, _vp]),
    "ssd_chunk_scan_fwd_static": (_i, [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _i, _i, _i, _i, _i, _i, _i, _i, _vp, _vp]),
    "ssd_selftest_bounded_wait": (_i, [_vp, ctypes.c_uint64, _vp]),
    "ssd_chunk_scan_varlen_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "ssd_chunk_scan_fwd_varlen": (_i, [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _i, _i, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp, _vp]),
    "ssd_conv_scan_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i, _i]),
    "ssd_decode_step": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                             _i, _i, _i, _i, _i, _i, _i, _vp]),
    "ssd_decode_step_workspace_bytes": (_sz, [_i, _i]),
    "ssd_decode_step_ws": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                _i, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp]),
    "ssd_chunk_scan_bwd_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "ssd_chunk_scan_bwd": (_i, [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                _i, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp]),
    "ssd_conv_scan_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                               _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp, _vp]),
    "ssd_linear_bf16": (_i, [_vp, _i64, _vp, _i64, _vp, _i64, _i, _i, _i, _vp, _vp]),
    "ssd_mixer_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i, _i, _i]),
    "ssd_mixer_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                           _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, ctypes.c_float, _i, _vp, _sz, _vp, _vp]),
}

# The entry points of include/ssd_diag.h.
DIAG_SIGNATURES = {
    "ssd_state_map_workspace_bytes": (_sz, [_i]),
    "ssd_state_map": (_i, [_vp] * 5 + [_i] * 6 + [_vp] * 8 + [_sz, _vp, _vp]),
    "ssd_conv1d_silu_varlen": (_i, [_vp, _i64, _vp, _i64] + [_vp] * 7 + [_i] * 7 + [_vp, _vp]),
    "ssd_conv1d_silu_bwd_workspace_bytes": (_sz, [_i] * 4),
    "ssd_conv1d_silu_bwd": (_i, [_vp] * 9 + [_i] * 5 + [_vp, _sz, _vp]),
    "ssd_diag_scan_workspace_bytes": (_sz, [_i] * 5),
    "ssd_diag_scan_fwd_workspace_bytes": (_sz, [_i] * 5),
    "ssd_diag_scan_fwd": (_i, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64] + [_vp] * 6 + [_i] * 6 + [_vp, _sz, _vp]),
    "ssd_diag_scan_fwd_varlen": (_i, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64] + [_vp] * 9 + [_i] * 8 +
                                 [_vp, _sz, _vp, _vp]),
    "ssd_diag_scan_bwd_workspace_bytes": (_sz, [_i] * 5),
    "ssd_diag_scan_bwd": (_i, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64] + [_vp] * 15 + [_i] * 6 + [_vp, _sz, _vp]),
    "ssd_diag_state_update": (_i, [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64] + [_vp] * 8 + [_i] * 8 + [_vp, _vp]),
}

_lock = threading.Lock()
_lib = None


class SsdError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


def load() -> ctypes.CDLL:
    """Load libssd.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"libssd.so not found at {LIB_PATH}: build it with "
                    "`python -m ssd_selective_scan_b200.build` (there is no fallback path)")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in (SIGNATURES | DIAG_SIGNATURES).items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def pycall_target() -> str:
    """The torch and Python whose headers the extension is built against: it
    reads tensors by their layout there."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def load_pycall():
    """The extension module of csrc/pycall.cpp.  Raises if it has not been
    built, or for another torch or Python."""
    load()
    try:
        from . import _pycall
    except ImportError as e:
        raise RuntimeError(f"{PYCALL_PATH}: {e}; build it with `python -m ssd_selective_scan_b200.build` (there is no fallback path)") from e
    built_for = getattr(_pycall, "built_for", "an unknown torch")
    if built_for != pycall_target():
        raise RuntimeError(f"{PYCALL_PATH} is built for {built_for}, this is {pycall_target()}: "
                           "build it with `python -m ssd_selective_scan_b200.build`")
    return _pycall


def status_string(status: int) -> str:
    return load().ssd_status_string(int(status)).decode()


def ssd_abi_version() -> int:
    return load().ssd_abi_version()


def ssd_conv1d_silu(xBC, out, w, bias, conv_state, b, L, conv_dim, k, dtype, stream) -> int:
    return load().ssd_conv1d_silu(xBC, out, w, bias, conv_state, b, L, conv_dim, k, dtype, stream)


def ssd_chunk_scan_workspace_bytes(b, L, H, P, N, G, Q, dtype) -> int:
    return load().ssd_chunk_scan_workspace_bytes(b, L, H, P, N, G, Q, dtype)


def ssd_chunk_scan_fwd(x, B, C, row_stride, dt_raw, dt_bias, A, D, init_state, y, final_state,
                       b, L, H, P, N, G, Q, dtype, workspace, workspace_bytes, status, stream) -> int:
    return load().ssd_chunk_scan_fwd(x, B, C, row_stride, dt_raw, dt_bias, A, D, init_state, y,
                                     final_state, b, L, H, P, N, G, Q, dtype, workspace,
                                     workspace_bytes, status, stream)


def ssd_chunk_scan_fwd_static(x, B, C, row_stride, dt_raw, dt_bias, A, D, init_state, y,
                              final_state, b, L, H, P, N, G, Q, dtype, status, stream) -> int:
    return load().ssd_chunk_scan_fwd_static(x, B, C, row_stride, dt_raw, dt_bias, A, D, init_state,
                                            y, final_state, b, L, H, P, N, G, Q, dtype, status,
                                            stream)


def ssd_state_update(state, x, B, C, row_stride, dt_raw, dt_bias, A, D, y, b, H, P, N, G, dtype,
                     stream) -> int:
    return load().ssd_state_update(state, x, B, C, row_stride, dt_raw, dt_bias, A, D, y, b, H, P,
                                   N, G, dtype, stream)


def ssd_chunk_scan_varlen_workspace_bytes(nseq, T, H, P, N, G, Q, dtype) -> int:
    return load().ssd_chunk_scan_varlen_workspace_bytes(nseq, T, H, P, N, G, Q, dtype)


def ssd_chunk_scan_fwd_varlen(x, B, C, row_stride, dt_raw, dt_bias, A, D, init_state, y, final_state,
                              cu_seqlens, nseq, T, H, P, N, G, Q, dtype, workspace, workspace_bytes,
                              status, stream) -> int:
    return load().ssd_chunk_scan_fwd_varlen(x, B, C, row_stride, dt_raw, dt_bias, A, D, init_state, y,
                                            final_state, cu_seqlens, nseq, T, H, P, N, G, Q, dtype,
                                            workspace, workspace_bytes, status, stream)


def ssd_conv_scan_workspace_bytes(b, L, H, P, N, G, Q, k, dtype) -> int:
    return load().ssd_conv_scan_workspace_bytes(b, L, H, P, N, G, Q, k, dtype)


def ssd_conv_scan_fwd(xBC, w, bias, conv_state, dt_raw, dt_bias, A, D, init_state, y, final_state,
                      b, L, H, P, N, G, Q, k, dtype, workspace, workspace_bytes, status, stream) -> int:
    return load().ssd_conv_scan_fwd(xBC, w, bias, conv_state, dt_raw, dt_bias, A, D, init_state, y,
                                    final_state, b, L, H, P, N, G, Q, k, dtype, workspace,
                                    workspace_bytes, status, stream)


def ssd_decode_step(state, conv_state, xBC, w, bias, dt_raw, dt_bias, A, D, y, b, H, P, N, G, k,
                    dtype, stream) -> int:
    return load().ssd_decode_step(state, conv_state, xBC, w, bias, dt_raw, dt_bias, A, D, y, b, H, P,
                                  N, G, k, dtype, stream)


def ssd_decode_step_workspace_bytes(b, G) -> int:
    return load().ssd_decode_step_workspace_bytes(b, G)


def ssd_decode_step_ws(state, conv_state, xBC, w, bias, dt_raw, dt_bias, A, D, y, b, H, P, N, G, k,
                       dtype, workspace, workspace_bytes, stream) -> int:
    return load().ssd_decode_step_ws(state, conv_state, xBC, w, bias, dt_raw, dt_bias, A, D, y, b, H, P,
                                     N, G, k, dtype, workspace, workspace_bytes, stream)


def ssd_chunk_scan_bwd_workspace_bytes(b, L, H, P, N, G, dtype) -> int:
    return load().ssd_chunk_scan_bwd_workspace_bytes(b, L, H, P, N, G, dtype)


def ssd_chunk_scan_bwd(x, B, C, row_stride, dt_raw, dt_bias, A, D, init_state, dy, dfinal, dx, dB, dC,
                       ddt_raw, dA, dD, ddt_bias, dinit, b, L, H, P, N, G, dtype, workspace,
                       workspace_bytes, stream) -> int:
    return load().ssd_chunk_scan_bwd(x, B, C, row_stride, dt_raw, dt_bias, A, D, init_state, dy, dfinal,
                                     dx, dB, dC, ddt_raw, dA, dD, ddt_bias, dinit, b, L, H, P, N, G,
                                     dtype, workspace, workspace_bytes, stream)


def ssd_selftest_bounded_wait(status, limit_ns, stream) -> int:
    return load().ssd_selftest_bounded_wait(status, limit_ns, stream)


def check(fn: str, status: int) -> None:
    if status != SSD_OK:
        raise SsdError(fn, status)


def ssd_linear_bf16(x, ldx, w, ldw, y, ldy, M, N, K, status, stream) -> int:
    return load().ssd_linear_bf16(x, ldx, w, ldw, y, ldy, M, N, K, status, stream)


def ssd_mixer_workspace_bytes(b, L, d_model, H, P, N, G, Q, k, dtype) -> int:
    return load().ssd_mixer_workspace_bytes(b, L, d_model, H, P, N, G, Q, k, dtype)


def ssd_mixer_fwd(hidden, W_in, conv_w, conv_bias, conv_state, dt_bias, A, D, norm_w, W_out, init_state, out,
                  final_state, b, L, d_model, H, P, N, G, Q, k, norm_groups, eps, dtype, workspace,
                  workspace_bytes, status, stream) -> int:
    return load().ssd_mixer_fwd(hidden, W_in, conv_w, conv_bias, conv_state, dt_bias, A, D, norm_w, W_out,
                                init_state, out, final_state, b, L, d_model, H, P, N, G, Q, k, norm_groups, eps,
                                dtype, workspace, workspace_bytes, status, stream)


def ssd_state_map_workspace_bytes(n) -> int:
    return load().ssd_state_map_workspace_bytes(n)


def ssd_state_map(lens, ctx, table, free_list, free_head, n, max_blocks, nfree, T, block_tokens, nslots, cu_seqlens,
                  seq_of, pos_of, slot_of, init_slot, table_out, free_head_out, workspace, workspace_bytes, status,
                  stream) -> int:
    return load().ssd_state_map(lens, ctx, table, free_list, free_head, n, max_blocks, nfree, T, block_tokens, nslots,
                                cu_seqlens, seq_of, pos_of, slot_of, init_slot, table_out, free_head_out, workspace,
                                workspace_bytes, status, stream)


def ssd_conv1d_silu_varlen(x, x_stride, out, out_stride, w, bias, cache, cu_seqlens, seq_of, slot_of, init_slot, nseq, T,
                           E, k, block_tokens, nslots, dtype, status, stream) -> int:
    return load().ssd_conv1d_silu_varlen(x, x_stride, out, out_stride, w, bias, cache, cu_seqlens, seq_of, slot_of,
                                         init_slot, nseq, T, E, k, block_tokens, nslots, dtype, status, stream)


def ssd_conv1d_silu_bwd_workspace_bytes(b, L, E, k) -> int:
    return load().ssd_conv1d_silu_bwd_workspace_bytes(b, L, E, k)


def ssd_conv1d_silu_bwd(x, w, bias, conv_state, dout, dx, dw, dbias, dconv_state, b, L, E, k, dtype, workspace,
                        workspace_bytes, stream) -> int:
    return load().ssd_conv1d_silu_bwd(x, w, bias, conv_state, dout, dx, dw, dbias, dconv_state, b, L, E, k, dtype,
                                      workspace, workspace_bytes, stream)


def ssd_diag_scan_workspace_bytes(nseq, rows, E, N, G) -> int:
    return load().ssd_diag_scan_workspace_bytes(nseq, rows, E, N, G)


def ssd_diag_scan_fwd_workspace_bytes(b, L, E, N, G) -> int:
    return load().ssd_diag_scan_fwd_workspace_bytes(b, L, E, N, G)


def ssd_diag_scan_fwd(u, u_stride, dt_raw, dt_stride, z, z_stride, B, C, bc_stride, A, dt_bias, D, init_state, y,
                      final_state, b, L, E, N, G, dtype, workspace, workspace_bytes, stream) -> int:
    return load().ssd_diag_scan_fwd(u, u_stride, dt_raw, dt_stride, z, z_stride, B, C, bc_stride, A, dt_bias, D,
                                    init_state, y, final_state, b, L, E, N, G, dtype, workspace, workspace_bytes, stream)


def ssd_diag_scan_fwd_varlen(u, u_stride, dt_raw, dt_stride, z, z_stride, B, C, bc_stride, A, dt_bias, D, states, y,
                             cu_seqlens, seq_of, slot_of, init_slot, nseq, T, E, N, G, block_tokens, nslots, dtype,
                             workspace, workspace_bytes, status, stream) -> int:
    return load().ssd_diag_scan_fwd_varlen(u, u_stride, dt_raw, dt_stride, z, z_stride, B, C, bc_stride, A, dt_bias, D,
                                           states, y, cu_seqlens, seq_of, slot_of, init_slot, nseq, T, E, N, G,
                                           block_tokens, nslots, dtype, workspace, workspace_bytes, status, stream)


def ssd_diag_scan_bwd_workspace_bytes(b, L, E, N, G) -> int:
    return load().ssd_diag_scan_bwd_workspace_bytes(b, L, E, N, G)


def ssd_diag_scan_bwd(u, u_stride, dt_raw, dt_stride, z, z_stride, B, C, bc_stride, A, dt_bias, D, init_state, dy, dfinal, du,
                      ddt_raw, dz, dB, dC, dA, dD, ddt_bias, dinit, b, L, E, N, G, dtype, workspace, workspace_bytes,
                      stream) -> int:
    return load().ssd_diag_scan_bwd(u, u_stride, dt_raw, dt_stride, z, z_stride, B, C, bc_stride, A, dt_bias, D, init_state,
                                    dy, dfinal, du, ddt_raw, dz, dB, dC, dA, dD, ddt_bias, dinit, b, L, E, N, G, dtype,
                                    workspace, workspace_bytes, stream)


def ssd_diag_state_update(states, u, u_stride, dt_raw, dt_stride, z, z_stride, B, C, bc_stride, A, dt_bias, D, y,
                          cu_seqlens, seq_of, slot_of, init_slot, nseq, rows, E, N, G, block_tokens, nslots, dtype, status,
                          stream) -> int:
    return load().ssd_diag_state_update(states, u, u_stride, dt_raw, dt_stride, z, z_stride, B, C, bc_stride, A, dt_bias,
                                        D, y, cu_seqlens, seq_of, slot_of, init_slot, nseq, rows, E, N, G, block_tokens,
                                        nslots, dtype, status, stream)
