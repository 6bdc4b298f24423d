"""Torch-facing calls of the diagonal selective scan (include/ssd_diag.h): the
state map of a batch of requests, the packed short conv and the conv's
gradient, the scan (dense, packed, backward) and the single-token update.

As in ``layer``, each function checks its tensors, allocates what it was not
given, passes raw pointers to the C entry point of the same name and raises
``SsdError`` on any non-OK status.  Work runs on the current stream of the
tensors' device, or on ``stream``.

A serving step with these calls::

    m = state_map(lens, ctx, table, free_list, free_head, T, block_tokens, nslots, status=status)
    u = conv1d_silu_varlen(x, conv_w, conv_cache, m, bias=conv_bias, status=status)
    dt_raw, B, C = projections of u
    y = diag_scan_fwd_varlen(u, dt_raw, A, B, C, states, m, dt_bias=dt_bias, D=D, z=z, status=status)

(``diag_state_update`` in the last line's place where every request brings one
token); ``status`` is read by the caller after synchronising, and 0 means that
every check on the device passed.  The calls do not wait for the device, so
nothing else tells: without a ``status`` (or with one that is not read) a batch
that a check refuses looks like an empty one, its outputs not written.

With ``stream``, results are the caller's to use on either stream.  Inputs, and
an ``out``, ``y`` or ``workspace`` that was given, have to be ready on that
stream, and to live until its work on them is done (``Tensor.record_stream``).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as libssd
from .layer import _dtype_code, _ptr

# The extension that checks the tensors and makes the calls (csrc/pycall.cpp),
# loaded with the first call; and its checks of a contiguous tensor, of evenly
# spaced rows and of B and C, each giving what the call takes.
_native = _dense = _rows = _bc = None


def _load():
    global _native, _dense, _rows, _bc
    ext = libssd.load_pycall()
    _dense, _rows, _bc = ext.dense, ext.rows, ext.bc
    _native = ext     # last: it tells another thread that the checks are there


class StateMap(NamedTuple):
    """Where a packed batch's requests, rows and states are (device tensors;
    the layouts are ssd_diag.h's).  The packed calls read cu_seqlens, seq_of,
    slot_of and init_slot; table and free_head are the scheduler's for the
    next step."""
    cu_seqlens: torch.Tensor          # [n + 1] int32
    seq_of: torch.Tensor              # [T] int32
    pos_of: torch.Tensor | None       # [T] int32
    slot_of: torch.Tensor             # [T] int64
    init_slot: torch.Tensor           # [n] int32
    table: torch.Tensor | None        # [n, max_blocks] int32
    free_head: torch.Tensor | None    # [1] int32
    block_tokens: int


class _On:
    """The device and stream of a call: the tensors' device is made current
    for it, and what the call allocates comes from the memory of `stream`
    where that is not the current one (a block that was freed on the current
    one may still be in use there).  (The current stream is asked for by its raw handle: a
    Stream object would cost as much host time as the launch.)"""
    __slots__ = ("device", "handle", "other", "switch", "scratch", "unread")

    def __init__(self, like: torch.Tensor, stream):
        if not like.is_cuda:
            raise ValueError("CUDA tensors expected")
        if _native is None:
            _load()
        self.device, self.handle, current = _native.where(like)
        self.switch = None if current else torch.cuda.device(self.device)
        self.other = None
        if stream is not None:
            if stream.device != self.device:
                raise ValueError("stream and tensors are on different devices")
            if stream.cuda_stream != self.handle:
                self.handle, self.other = stream.cuda_stream, stream

    def __enter__(self):
        if self.switch is not None:
            self.switch.__enter__()
        return self

    def __exit__(self, *exc):
        if self.switch is not None:
            self.switch.__exit__(*exc)

    def empty(self, shape, dtype):
        if self.other is None:
            return _native.empty(shape, dtype, self.device)
        with torch.cuda.stream(self.other):
            t = _native.empty(shape, dtype, self.device)
        # and the caller may use it here up to the moment it is freed
        t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def map_out(self, n, max_blocks, T, extra):
        """A new map's tensors, and the address of `extra` more int32."""
        if self.other is None:
            return _native.map_out(n, max_blocks, T, extra, self.device)
        with torch.cuda.stream(self.other):
            made = _native.map_out(n, max_blocks, T, extra, self.device)
        for t in made[:-1]:
            t.record_stream(torch.cuda.current_stream(self.device))
        return made

    def workspace(self, given, need: int):
        """(pointer, bytes) of the caller's workspace, or of a new one."""
        if given is None:
            if not need:
                return None, 0
            given = self.scratch = self.empty((need,), torch.uint8)
        elif given.device != self.device or not given.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {self.device}")
        return given.data_ptr(), given.numel() * given.element_size()


def _map(m: StateMap, T: int, device):
    """The pointers of a StateMap, its requests and block size."""
    return _native.map_in(m[0], m[1], m[3], m[4], T, device)


def _status(status, on):
    if status is None:
        # of the call's own: nobody reads it, but the kernels need the place
        status = on.unread = on.empty((1,), torch.int32)
    return _dense(status, "status", torch.int32, (1,), on.device)


def state_map(lens: torch.Tensor, ctx: torch.Tensor, table: torch.Tensor, free_list: torch.Tensor, free_head: torch.Tensor,
              T: int, block_tokens: int, nslots: int, *, out: StateMap | None = None, workspace: torch.Tensor | None = None,
              status: torch.Tensor | None = None, stream=None) -> StateMap:
    """The map of a batch of requests: lens, ctx [n] int32 (new and held
    tokens), table [n, max_blocks] int32 (slots of the held blocks), free_list
    [nfree] and free_head [1] int32; T rows in the packed batch.  Returns a
    StateMap whose table and free_head are the updated ones (new tensors, or
    `out`'s, which may be the inputs for an update in place; `out` is for n
    requests, T rows and this block size).  A batch that
    does not fit (ssd_diag.h) leaves SSD_ERR_INVALID_ARG in `status` and gives
    an empty map."""
    n = lens.numel()
    i32 = torch.int32
    if table.dim() != 2 or table.shape[0] != n:
        raise ValueError("table must be [n, max_blocks]")
    mb = table.shape[1]
    if out is not None and out.block_tokens != block_tokens:
        raise ValueError("out was made for another block size")
    with _On(lens, stream) as on:
        dev = on.device
        scratch = 64 + n      # the workspace, in int32
        if out is None:
            *parts, end = on.map_out(n, mb, T, 0 if workspace is not None else scratch)
            out = StateMap(*parts, block_tokens)
            ptrs = [t.data_ptr() for t in parts]
            if workspace is None:
                wp, wb = end, 4 * scratch
        else:
            cu, seq, slot, init, made_for = _map(out, T, dev)
            if made_for != n:   # its tensors would be written past their ends, or keep old requests
                raise ValueError(f"out is the map of {made_for} requests, lens of {n}")
            ptrs = (cu, seq, _dense(out.pos_of, "pos_of", i32, (T,), dev), slot, init, _dense(out.table, "out.table", i32, (n, mb), dev),
                    _dense(out.free_head, "out.free_head", i32, (1,), dev))
            if workspace is None:
                wp, wb = on.workspace(None, 4 * scratch)
        if workspace is not None:
            wp, wb = on.workspace(workspace, 4 * scratch)
        nfree = free_list.numel()
        st = _native.ssd_state_map(
            _dense(lens, "lens", i32, (n,), dev), _dense(ctx, "ctx", i32, (n,), dev), _dense(table, "table", i32, (n, mb), dev),
            _dense(free_list, "free_list", i32, (nfree,), dev), _dense(free_head, "free_head", i32, (1,), dev),
            n, mb, nfree, T, block_tokens, nslots, *ptrs, wp, wb, _status(status, on), on.handle)
        libssd.check("ssd_state_map", st)
    return out


def conv1d_silu_varlen(x: torch.Tensor, w: torch.Tensor, cache: torch.Tensor, m: StateMap, *, bias: torch.Tensor | None = None,
                       out: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal depthwise conv1d + SiLU over packed requests.  x [T, E] (dense
    rows at any stride); w [E, k] f32; cache [nslots, E, k] of x's dtype,
    read and written by slot.  Returns out [T, E]; rows behind the last
    request are left as they were."""
    if x.dim() != 2:
        raise ValueError("x must be [T, E]")
    T, E = x.shape
    k = w.shape[-1]
    with _On(x, stream) as on:
        dev = on.device
        if out is None:
            out = on.empty((T, E), x.dtype)
        xp, xs = _rows(x, "x", (T,), E, x)
        op, os_ = _rows(out, "out", (T,), E, x)
        cu, seq, slot, init, n = _map(m, T, dev)
        nslots = cache.shape[0]
        st = _native.ssd_conv1d_silu_varlen(xp, xs, op, os_, _dense(w, "w", torch.float32, (E, k), dev),
                                            _dense(bias, "bias", torch.float32, (E,), dev),
                                            _dense(cache, "cache", x.dtype, (nslots, E, k), dev), cu, seq, slot, init, n, T, E, k,
                                            m.block_tokens, nslots, _dtype_code(x), _status(status, on), on.handle)
        libssd.check("ssd_conv1d_silu_varlen", st)
    return out


def conv1d_silu_bwd(x: torch.Tensor, w: torch.Tensor, dout: torch.Tensor, bias: torch.Tensor | None = None,
                    conv_state: torch.Tensor | None = None, *, workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Gradients through conv1d_silu.  x, dout [b, L, E]; w [E, k] f32, bias
    [E] f32, conv_state [b, E, k] (the cache as the forward call found it).
    Returns dict(dx, dw, dbias, dconv_state): dx and dconv_state in the I/O
    dtype, dw and dbias f32; None for what the forward call did not have."""
    if x.dim() != 3:
        raise ValueError("x must be [b, L, E]")
    b, L, E = x.shape
    k = w.shape[-1]
    f32 = torch.float32
    with _On(x, stream) as on:
        dev = on.device
        r = dict(dx=on.empty((b, L, E), x.dtype), dw=on.empty((E, k), f32), dbias=None if bias is None else on.empty((E,), f32),
                 dconv_state=None if conv_state is None else on.empty((b, E, k), x.dtype))
        wp, wb = on.workspace(workspace, _native.ssd_conv1d_silu_bwd_workspace_bytes(b, L, E, k))
        st = _native.ssd_conv1d_silu_bwd(_dense(x, "x", x.dtype, (b, L, E), dev), _dense(w, "w", f32, (E, k), dev),
                                         _dense(bias, "bias", f32, (E,), dev), _dense(conv_state, "conv_state", x.dtype, (b, E, k), dev),
                                         _dense(dout, "dout", x.dtype, (b, L, E), dev), _ptr(r["dx"]), _ptr(r["dw"]), _ptr(r["dbias"]),
                                         _ptr(r["dconv_state"]), b, L, E, k, _dtype_code(x), wp, wb, on.handle)
        libssd.check("ssd_conv1d_silu_bwd", st)
    return r


def diag_scan_workspace_bytes(nseq: int, rows: int, E: int, N: int, G: int) -> int:
    """Workspace of diag_scan_fwd_varlen (rows = T), and enough for
    diag_scan_fwd (nseq = b, rows = b * L; none where its sequences are not
    cut: ssd_diag.h)."""
    return int(libssd.ssd_diag_scan_workspace_bytes(nseq, rows, E, N, G))


def diag_scan_fwd(u: torch.Tensor, dt_raw: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, *,
                  dt_bias: torch.Tensor | None = None, D: torch.Tensor | None = None, z: torch.Tensor | None = None,
                  init_state: torch.Tensor | None = None, y: torch.Tensor | None = None,
                  final_state: torch.Tensor | bool | None = True, workspace: torch.Tensor | None = None, stream=None):
    """The diagonal scan of a dense batch.  u, dt_raw, z [b, L, E], B, C
    [b, L, G, N] (views with dense rows at any stride), A [E, N] f32, dt_bias,
    D [E] f32, init_state [b, E, N] f32.  Returns (y [b, L, E], final_state
    [b, E, N] f32 or None)."""
    if u.dim() != 3:
        raise ValueError("u must be [b, L, E]")
    b, L, E = u.shape
    f32 = torch.float32
    with _On(u, stream) as on:
        dev = on.device
        pB, pC, bcs, G, N = _bc(B, C, (b, L), u)
        if y is None:
            y = on.empty((b, L, E), u.dtype)
        if final_state is True:
            final_state = on.empty((b, E, N), f32)
        elif final_state is False:
            final_state = None
        up, us = _rows(u, "u", (b, L), E, u)
        dp, ds = _rows(dt_raw, "dt_raw", (b, L), E, u)
        zp, zs = _rows(z, "z", (b, L), E, u)
        wp, wb = on.workspace(workspace, _native.ssd_diag_scan_fwd_workspace_bytes(b, L, E, N, G))
        st = _native.ssd_diag_scan_fwd(up, us, dp, ds, zp, zs, pB, pC, bcs, _dense(A, "A", f32, (E, N), dev),
                                       _dense(dt_bias, "dt_bias", f32, (E,), dev), _dense(D, "D", f32, (E,), dev),
                                       _dense(init_state, "init_state", f32, (b, E, N), dev), _dense(y, "y", u.dtype, (b, L, E), dev),
                                       _dense(final_state, "final_state", f32, (b, E, N), dev), b, L, E, N, G, _dtype_code(u), wp, wb,
                                       on.handle)
        libssd.check("ssd_diag_scan_fwd", st)
    return y, final_state


def diag_scan_fwd_varlen(u: torch.Tensor, dt_raw: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                         states: torch.Tensor, m: StateMap, *, dt_bias: torch.Tensor | None = None, D: torch.Tensor | None = None,
                         z: torch.Tensor | None = None, y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The diagonal scan of packed requests.  u, dt_raw, z [T, E], B, C
    [T, G, N]; states [nslots, E, N] f32, read and written by slot.  Returns y
    [T, E]; rows behind the last request are left as they were."""
    if u.dim() != 2:
        raise ValueError("u must be [T, E]")
    T, E = u.shape
    f32 = torch.float32
    with _On(u, stream) as on:
        dev = on.device
        pB, pC, bcs, G, N = _bc(B, C, (T,), u)
        if y is None:
            y = on.empty((T, E), u.dtype)
        up, us = _rows(u, "u", (T,), E, u)
        dp, ds = _rows(dt_raw, "dt_raw", (T,), E, u)
        zp, zs = _rows(z, "z", (T,), E, u)
        cu, seq, slot, init, n = _map(m, T, dev)
        nslots = states.shape[0]
        wp, wb = on.workspace(workspace, _native.ssd_diag_scan_workspace_bytes(n, T, E, N, G))
        st = _native.ssd_diag_scan_fwd_varlen(up, us, dp, ds, zp, zs, pB, pC, bcs, _dense(A, "A", f32, (E, N), dev),
                                              _dense(dt_bias, "dt_bias", f32, (E,), dev), _dense(D, "D", f32, (E,), dev),
                                              _dense(states, "states", f32, (nslots, E, N), dev), _dense(y, "y", u.dtype, (T, E), dev),
                                              cu, seq, slot, init, n, T, E, N, G, m.block_tokens, nslots, _dtype_code(u), wp, wb,
                                              _status(status, on), on.handle)
        libssd.check("ssd_diag_scan_fwd_varlen", st)
    return y


def diag_scan_bwd(u: torch.Tensor, dt_raw: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, dy: torch.Tensor, *,
                  dt_bias: torch.Tensor | None = None, D: torch.Tensor | None = None, z: torch.Tensor | None = None,
                  init_state: torch.Tensor | None = None, dfinal: torch.Tensor | None = None, want_dinit: bool = True,
                  workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Gradients through diag_scan_fwd.  Inputs as for the forward call; dy
    [b, L, E] (I/O dtype), dfinal [b, E, N] f32 or None.  Returns dict(du,
    ddt_raw, dz, dB, dC, dA, dD, ddt_bias, dinit): du, ddt_raw, dz [b, L, E]
    and dB, dC [b, L, G, N] in the I/O dtype, the others f32; dz is None
    without z, dinit if not wanted."""
    if u.dim() != 3:
        raise ValueError("u must be [b, L, E]")
    b, L, E = u.shape
    f32 = torch.float32
    with _On(u, stream) as on:
        dev = on.device
        pB, pC, bcs, G, N = _bc(B, C, (b, L), u)
        up, us = _rows(u, "u", (b, L), E, u)
        dp, ds = _rows(dt_raw, "dt_raw", (b, L), E, u)
        zp, zs = _rows(z, "z", (b, L), E, u)
        io, bc = (lambda: on.empty((b, L, E), u.dtype)), (lambda: on.empty((b, L, G, N), u.dtype))
        r = dict(du=io(), ddt_raw=io(), dz=None if z is None else io(), dB=bc(), dC=bc(), dA=on.empty((E, N), f32), dD=on.empty((E,), f32),
                 ddt_bias=on.empty((E,), f32), dinit=on.empty((b, E, N), f32) if want_dinit else None)
        wp, wb = on.workspace(workspace, _native.ssd_diag_scan_bwd_workspace_bytes(b, L, E, N, G))
        st = _native.ssd_diag_scan_bwd(up, us, dp, ds, zp, zs, pB, pC, bcs, _dense(A, "A", f32, (E, N), dev),
                                       _dense(dt_bias, "dt_bias", f32, (E,), dev), _dense(D, "D", f32, (E,), dev),
                                       _dense(init_state, "init_state", f32, (b, E, N), dev), _dense(dy, "dy", u.dtype, (b, L, E), dev),
                                       _dense(dfinal, "dfinal", f32, (b, E, N), dev), _ptr(r["du"]), _ptr(r["ddt_raw"]), _ptr(r["dz"]),
                                       _ptr(r["dB"]), _ptr(r["dC"]), _ptr(r["dA"]), _ptr(r["dD"]), _ptr(r["ddt_bias"]), _ptr(r["dinit"]),
                                       b, L, E, N, G, _dtype_code(u), wp, wb, on.handle)
        libssd.check("ssd_diag_scan_bwd", st)
    return r


def diag_state_update(states: torch.Tensor, u: torch.Tensor, dt_raw: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                      C: torch.Tensor, m: StateMap | None = None, *, dt_bias: torch.Tensor | None = None,
                      D: torch.Tensor | None = None, z: torch.Tensor | None = None, y: torch.Tensor | None = None,
                      status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One token per request, states [nslots, E, N] f32 updated in place by
    slot (without a map row i is state i).  u, dt_raw, z [rows, E], B, C
    [rows, G, N].  Returns y [rows, E]."""
    if u.dim() != 2:
        raise ValueError("u must be [rows, E]")
    T, E = u.shape
    f32 = torch.float32
    with _On(u, stream) as on:
        dev = on.device
        pB, pC, bcs, G, N = _bc(B, C, (T,), u)
        if y is None:
            y = on.empty((T, E), u.dtype)
        up, us = _rows(u, "u", (T,), E, u)
        dp, ds = _rows(dt_raw, "dt_raw", (T,), E, u)
        zp, zs = _rows(z, "z", (T,), E, u)
        cu = seq = slot = init = sp = None
        n, bs = 0, 1
        if m is not None:
            cu, seq, slot, init, n = _map(m, T, dev)
            bs = m.block_tokens
            sp = _status(status, on)
        nslots = states.shape[0]
        st = _native.ssd_diag_state_update(_dense(states, "states", f32, (nslots, E, N), dev), up, us, dp, ds, zp, zs, pB, pC, bcs,
                                           _dense(A, "A", f32, (E, N), dev), _dense(dt_bias, "dt_bias", f32, (E,), dev),
                                           _dense(D, "D", f32, (E,), dev), _dense(y, "y", u.dtype, (T, E), dev), cu, seq, slot, init, n,
                                           T, E, N, G, bs, nslots, _dtype_code(u), sp, on.handle)
        libssd.check("ssd_diag_state_update", st)
    return y
