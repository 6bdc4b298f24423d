"""B200-native (sm_100a) hot path of the Mamba-2 selective state-space layer.

libssd.so (built from csrc/ by ``python -m ssd_selective_scan_b200.build``)
holds the CUDA kernels behind the C ABI of include/ssd.h and
include/ssd_diag.h; ``binding`` is its ctypes binding, ``layer`` the
torch-facing calls and ``diag`` those of the diagonal selective scan, which go
through the extension _pycall.so (csrc/pycall.cpp).  Both are loaded on first
use and there is no fallback path: without them every call raises.
"""
from .layer import (chunk_scan_bwd, chunk_scan_bwd_workspace_bytes, chunk_scan_fwd, chunk_scan_fwd_varlen, chunk_scan_varlen_workspace_bytes,
                    chunk_scan_workspace_bytes, conv1d_silu, conv_scan_fwd, conv_scan_workspace_bytes,
                    decode_step, layer_prefill, split_channels, state_update)
from .diag import (StateMap, conv1d_silu_bwd, conv1d_silu_varlen, diag_scan_bwd, diag_scan_fwd, diag_scan_fwd_varlen, diag_scan_workspace_bytes,
                   diag_state_update, state_map)
from .binding import SsdError

__all__ = ["chunk_scan_bwd", "chunk_scan_bwd_workspace_bytes", "chunk_scan_fwd", "chunk_scan_fwd_varlen", "chunk_scan_varlen_workspace_bytes",
           "chunk_scan_workspace_bytes", "conv1d_silu", "conv_scan_fwd", "conv_scan_workspace_bytes",
           "decode_step", "StateMap", "conv1d_silu_bwd", "conv1d_silu_varlen", "diag_scan_bwd", "diag_scan_fwd", "diag_scan_fwd_varlen",
           "diag_scan_workspace_bytes", "diag_state_update", "state_map",
           "layer_prefill", "split_channels", "state_update", "SsdError"]
