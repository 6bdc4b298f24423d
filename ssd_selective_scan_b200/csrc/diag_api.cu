// diag_api.cu -- the extern "C" entry points declared in include/ssd_diag.h:
// argument validation, kernel launch.  No allocation, no synchronisation, no
// global mutable state.
#include "ssd_diag.h"

#include <initializer_list>

#include "abi.h"
#include "diag.h"

namespace {

using namespace ssd;

// A tensor of `rows` rows of `width` elements of e bytes at a row stride.
Range rows_span(const void* p, int64_t rows, int64_t stride, int64_t width, int e)
{
    return span(p, p && rows > 0 ? ((rows - 1) * stride + width) * e : 0);
}

// Whether one of the written ranges overlaps a read one or another written one.
bool clash(std::initializer_list<Range> written, std::initializer_list<Range> read)
{
    for (const Range* w = written.begin(); w != written.end(); ++w) {
        for (const Range& r : read)
            if (overlap(*w, r)) return true;
        for (const Range* v = w + 1; v != written.end(); ++v)
            if (overlap(*w, *v)) return true;
    }
    return false;
}

bool all_aligned(std::initializer_list<const void*> ptrs, uintptr_t n)
{
    for (const void* p : ptrs)
        if (p && !aligned(p, n)) return false;
    return true;
}

// The sizes, strides and pointers that the scan calls share; SSD_OK if sound.
ssd_status_t check_scan(const DiagArgs& a, ssd_dtype_t dtype)
{
    if (!valid_dtype(dtype) || a.nseq < 0 || a.L < 0 || a.rows < 0 || a.E <= 0 || a.N <= 0 || a.G <= 0) return SSD_ERR_INVALID_ARG;
    if (a.E % a.G || (a.E / a.G) % 8 || a.N % 4) return SSD_ERR_INVALID_ARG;
    if (!a.A || !all_aligned({a.A, a.init, a.final_state}, 16) || !all_aligned({a.dt_bias, a.D}, 4)) return SSD_ERR_INVALID_ARG;
    if (a.rows > 0) {
        if (!a.u || !a.dt || !a.B || !a.C) return SSD_ERR_INVALID_ARG;
        if (!all_aligned({a.u, a.dt, a.z, a.y}, 16) || !all_aligned({a.B, a.C}, elem_bytes(dtype))) return SSD_ERR_INVALID_ARG;
        for (const int64_t st : {a.us, a.dts, a.z ? a.zs : a.us})
            if (st % 8 || st < a.E) return SSD_ERR_INVALID_ARG;
        if (a.bcs < (int64_t)a.G * a.N) return SSD_ERR_INVALID_ARG;
    }
    if (a.N > 64) return SSD_ERR_UNSUPPORTED;
    if ((int64_t)a.E / 8 + a.G > 65535) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

struct ScanRanges {
    Range u, dt, z, B, C, y, A, bias, D;
};
ScanRanges scan_ranges(const DiagArgs& a, int e)
{
    const int64_t bc = (int64_t)a.G * a.N;
    return ScanRanges{rows_span(a.u, a.rows, a.us, a.E, e), rows_span(a.dt, a.rows, a.dts, a.E, e),
                      rows_span(a.z, a.rows, a.zs, a.E, e), rows_span(a.B, a.rows, a.bcs, bc, e),
                      rows_span(a.C, a.rows, a.bcs, bc, e), rows_span(a.y, a.rows, a.E, a.E, e),
                      span(a.A, (int64_t)a.E * a.N * 4), span(a.dt_bias, a.dt_bias ? (int64_t)a.E * 4 : 0),
                      span(a.D, a.D ? (int64_t)a.E * 4 : 0)};
}

struct MapRanges {
    Range cu, seq, slot, init, status;
};
MapRanges map_ranges(const SlotArgs& s, int rows)
{
    return MapRanges{span(s.cu, s.cu ? (int64_t)(s.nseq + 1) * 4 : 0), span(s.seq_of, s.cu ? (int64_t)rows * 4 : 0),
                     span(s.slot_of, s.cu ? (int64_t)rows * 8 : 0), span(s.init_slot, s.cu ? (int64_t)s.nseq * 4 : 0),
                     span(s.status, s.status ? 4 : 0)};
}

// A packed call's map: present, aligned, of sound sizes.
ssd_status_t check_map(const SlotArgs& s, int T)
{
    if (s.nseq < 0 || s.nslots < 0 || s.block <= 0) return SSD_ERR_INVALID_ARG;
    if (!s.cu || !s.status || (T > 0 && (!s.seq_of || !s.slot_of)) || (s.nseq > 0 && !s.init_slot)) return SSD_ERR_INVALID_ARG;
    if (!all_aligned({s.cu, s.seq_of, s.init_slot, s.status}, 4) || !all_aligned({s.slot_of}, 8)) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

}  // namespace

extern "C" {

size_t ssd_state_map_workspace_bytes(int n)
{
    return n < 0 ? 0 : ((size_t)kMapWsHeader + n) * 4;
}

ssd_status_t ssd_state_map(const int32_t* lens, const int32_t* ctx, const int32_t* table, const int32_t* free_list,
                           const int32_t* free_head, int n, int max_blocks, int nfree, int T, int block_tokens,
                           int nslots, int32_t* cu_seqlens, int32_t* seq_of, int32_t* pos_of, int64_t* slot_of,
                           int32_t* init_slot, int32_t* table_out, int32_t* free_head_out, void* workspace,
                           size_t workspace_bytes, int32_t* status, cudaStream_t stream)
{
    if (n < 0 || max_blocks < 0 || nfree < 0 || T < 0 || block_tokens <= 0 || nslots < 0) return SSD_ERR_INVALID_ARG;
    if (!free_head || !free_head_out || !cu_seqlens || !status || !workspace ||
        workspace_bytes < ssd_state_map_workspace_bytes(n))
        return SSD_ERR_INVALID_ARG;
    if (n > 0 && (!lens || !ctx || !init_slot || (max_blocks > 0 && (!table || !table_out)))) return SSD_ERR_INVALID_ARG;
    if ((nfree > 0 && !free_list) || (T > 0 && (!seq_of || !pos_of || !slot_of))) return SSD_ERR_INVALID_ARG;
    if (!all_aligned({lens, ctx, table, free_list, free_head, cu_seqlens, init_slot, table_out, free_head_out, workspace, status}, 4) ||
        !all_aligned({seq_of, pos_of, slot_of}, 16))
        return SSD_ERR_INVALID_ARG;
    if (n > (1 << 24) || T > kMaxRows || (int64_t)n * max_blocks > 0x7fffffffLL || nslots > kMapMaxSlots) return SSD_ERR_UNSUPPORTED;
    const int64_t entries = (int64_t)n * max_blocks;
    const Range table_in = span(table, entries * 4), table_o = span(table_out, entries * 4);
    const Range head_in = span(free_head, 4), head_o = span(free_head_out, 4);
    const Range in[] = {span(lens, (int64_t)n * 4), span(ctx, (int64_t)n * 4), span(free_list, (int64_t)nfree * 4)};
    const Range cu = span(cu_seqlens, (int64_t)(n + 1) * 4), seq = span(seq_of, (int64_t)T * 4), pos = span(pos_of, (int64_t)T * 4);
    const Range slot = span(slot_of, (int64_t)T * 8), init = span(init_slot, (int64_t)n * 4);
    const Range ws = span(workspace, (int64_t)workspace_bytes), st = span(status, 4);
    if (clash({cu, seq, pos, slot, init, table_o, head_o, ws, st}, {in[0], in[1], in[2]})) return SSD_ERR_INVALID_ARG;
    if (clash({cu, seq, pos, slot, init, ws, st}, {table_in, head_in})) return SSD_ERR_INVALID_ARG;
    if ((table_out != table && overlap(table_o, table_in)) || (free_head_out != free_head && overlap(head_o, head_in)) ||
        overlap(table_o, head_in) || overlap(head_o, table_in))
        return SSD_ERR_INVALID_ARG;
    StateMapArgs a{lens, ctx, table, free_list, free_head, n, max_blocks, nfree, T, block_tokens, nslots, cu_seqlens,
                   seq_of, pos_of, slot_of, init_slot, table_out, free_head_out, static_cast<int32_t*>(workspace), status};
    return from_cuda(launch_state_map(a, stream));
}

ssd_status_t ssd_conv1d_silu_varlen(const void* x, int64_t x_stride, void* out, int64_t out_stride, const float* w,
                                    const float* bias, void* cache, const int32_t* cu_seqlens, const int32_t* seq_of,
                                    const int64_t* slot_of, const int32_t* init_slot, int nseq, int T, int E, int k,
                                    int block_tokens, int nslots, ssd_dtype_t dtype, int32_t* status,
                                    cudaStream_t stream)
{
    if (!valid_dtype(dtype) || T < 0 || E <= 0 || E % 8 || k <= 0) return SSD_ERR_INVALID_ARG;
    const SlotArgs sl{cu_seqlens, seq_of, slot_of, init_slot, nseq, nslots, block_tokens, status};
    ssd_status_t st = check_map(sl, T);
    if (st != SSD_OK) return st;
    if (T > 0 && (!x || !out || !w || (nslots > 0 && !cache))) return SSD_ERR_INVALID_ARG;
    if (x_stride % 8 || x_stride < E || out_stride % 8 || out_stride < E) return SSD_ERR_INVALID_ARG;
    if (!all_aligned({x, out, cache, w}, 16) || !aligned(bias, 4)) return SSD_ERR_INVALID_ARG;
    const int e = elem_bytes(dtype);
    const MapRanges m = map_ranges(sl, T);
    if (clash({rows_span(out, T, out_stride, E, e), span(cache, (int64_t)nslots * E * k * e), m.status},
              {rows_span(x, T, x_stride, E, e), span(w, (int64_t)E * k * 4), span(bias, bias ? (int64_t)E * 4 : 0), m.cu, m.seq,
               m.slot, m.init}))
        return SSD_ERR_INVALID_ARG;
    if (k < 2 || k > 4 || E / 512 > 65534) return SSD_ERR_UNSUPPORTED;
    if ((int64_t)nseq + T > kMaxRows) return SSD_ERR_UNSUPPORTED;
    if (T == 0 || nseq == 0) return SSD_OK;
    return from_cuda(launch_conv1d_varlen(x, x_stride, out, out_stride, w, bias, cache, sl, T, E, k, dtype == SSD_BF16, stream));
}

size_t ssd_conv1d_silu_bwd_workspace_bytes(int b, int L, int E, int k)
{
    return b <= 0 || L <= 0 || (int64_t)b * L > kMaxRows || E <= 0 || k <= 0 ? 0 : conv1d_bwd_workspace_bytes(b, L, E, k);
}

ssd_status_t ssd_conv1d_silu_bwd(const void* x, const float* w, const float* bias, const void* conv_state,
                                 const void* dout, void* dx, float* dw, float* dbias, void* dconv_state, int b, int L,
                                 int E, int k, ssd_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                 cudaStream_t stream)
{
    if (!valid_dtype(dtype) || b < 0 || L < 0 || E <= 0 || E % 8 || k <= 0) return SSD_ERR_INVALID_ARG;
    const bool tokens = b > 0 && L > 0;
    if (!dw || (tokens && (!x || !w || !dout || !dx))) return SSD_ERR_INVALID_ARG;
    if (!all_aligned({x, dout, dx, conv_state, dconv_state, workspace, w}, 16) || !all_aligned({bias, dw, dbias}, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t need = ssd_conv1d_silu_bwd_workspace_bytes(b, L, E, k);
    if (workspace_bytes < need || (need && !workspace)) return SSD_ERR_INVALID_ARG;
    const int e = elem_bytes(dtype);
    const int64_t io = (int64_t)b * L * E * e, cache = (int64_t)b * E * k * e, wb = (int64_t)E * k * 4;
    if (clash({span(dx, io), span(dw, wb), span(dbias, dbias ? (int64_t)E * 4 : 0), span(dconv_state, dconv_state ? cache : 0),
               span(workspace, (int64_t)need)},
              {span(x, io), span(w, wb), span(bias, bias ? (int64_t)E * 4 : 0), span(conv_state, conv_state ? cache : 0), span(dout, io)}))
        return SSD_ERR_INVALID_ARG;
    if (k < 2 || k > 4 || E / 512 > 65534 || (int64_t)b * L > kMaxRows) return SSD_ERR_UNSUPPORTED;
    if (!tokens) {
        cudaError_t err = cudaMemsetAsync(dw, 0, (size_t)wb, stream);
        if (err == cudaSuccess && dbias) err = cudaMemsetAsync(dbias, 0, (size_t)E * 4, stream);
        if (err == cudaSuccess && dconv_state && b > 0) err = cudaMemsetAsync(dconv_state, 0, (size_t)cache, stream);
        return from_cuda(err);
    }
    return from_cuda(launch_conv1d_bwd(x, w, bias, conv_state, dout, dx, dw, dbias, dconv_state, b, L, E, k,
                                       dtype == SSD_BF16, workspace, stream));
}

size_t ssd_diag_scan_workspace_bytes(int nseq, int rows, int E, int N, int G)
{
    if (nseq <= 0 || rows <= 0 || E <= 0 || N <= 0 || N > 64 || G <= 0 || E % G) return 0;
    return diag_scan_workspace_bytes(nseq, rows, E, N, G);
}

size_t ssd_diag_scan_fwd_workspace_bytes(int b, int L, int E, int N, int G)
{
    if (b <= 0 || L <= 0 || (int64_t)b * L > kMaxRows || E <= 0 || N <= 0 || N > 64 || G <= 0 || E % G) return 0;
    return diag_scan_fwd_workspace_bytes(b, L, E, N, G);
}

ssd_status_t ssd_diag_scan_fwd(const void* u, int64_t u_stride, const void* dt_raw, int64_t dt_stride, const void* z,
                               int64_t z_stride, const void* B, const void* C, int64_t bc_stride, const float* A,
                               const float* dt_bias, const float* D, const float* init_state, void* y,
                               float* final_state, int b, int L, int E, int N, int G, ssd_dtype_t dtype,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    if (b < 0 || L < 0) return SSD_ERR_INVALID_ARG;
    if ((int64_t)b * L > kMaxRows) return SSD_ERR_UNSUPPORTED;
    DiagArgs a{u, dt_raw, z, B, C, u_stride, dt_stride, z_stride, bc_stride, A, dt_bias, D, init_state, y, final_state,
               b, L, b * L, E, N, G, dtype == SSD_BF16, SlotArgs{}, workspace};
    const ssd_status_t st = check_scan(a, dtype);
    if (st != SSD_OK) return st;
    if (a.rows > 0 && !y) return SSD_ERR_INVALID_ARG;
    const size_t need = ssd_diag_scan_fwd_workspace_bytes(b, L, E, N, G);
    if (workspace_bytes < need || (need && (!workspace || !aligned(workspace, 16)))) return SSD_ERR_INVALID_ARG;
    const ScanRanges r = scan_ranges(a, elem_bytes(dtype));
    const int64_t st_bytes = (int64_t)b * E * N * 4;
    const Range ri = span(init_state, init_state ? st_bytes : 0), rf = span(final_state, final_state ? st_bytes : 0);
    const Range rw = span(workspace, (int64_t)need);
    if (clash({r.y, rf, rw}, {r.u, r.dt, r.z, r.B, r.C, r.A, r.bias, r.D})) return SSD_ERR_INVALID_ARG;
    if (overlap(r.y, ri) || overlap(rw, ri) || (final_state != init_state && overlap(rf, ri))) return SSD_ERR_INVALID_ARG;
    if (b == 0) return SSD_OK;
    if (L == 0) {
        if (!final_state || final_state == init_state) return SSD_OK;
        return from_cuda(init_state ? cudaMemcpyAsync(final_state, init_state, (size_t)st_bytes, cudaMemcpyDeviceToDevice, stream)
                                    : cudaMemsetAsync(final_state, 0, (size_t)st_bytes, stream));
    }
    return from_cuda(launch_diag_scan(a, stream));
}

ssd_status_t ssd_diag_scan_fwd_varlen(const void* u, int64_t u_stride, const void* dt_raw, int64_t dt_stride,
                                      const void* z, int64_t z_stride, const void* B, const void* C,
                                      int64_t bc_stride, const float* A, const float* dt_bias, const float* D,
                                      float* states, void* y, const int32_t* cu_seqlens, const int32_t* seq_of,
                                      const int64_t* slot_of, const int32_t* init_slot, int nseq, int T, int E, int N,
                                      int G, int block_tokens, int nslots, ssd_dtype_t dtype, void* workspace,
                                      size_t workspace_bytes, int32_t* status, cudaStream_t stream)
{
    DiagArgs a{u, dt_raw, z, B, C, u_stride, dt_stride, z_stride, bc_stride, A, dt_bias, D, states, y, states,
               nseq, 0, T, E, N, G, dtype == SSD_BF16,
               SlotArgs{cu_seqlens, seq_of, slot_of, init_slot, nseq, nslots, block_tokens, status}, workspace};
    ssd_status_t st = check_scan(a, dtype);
    if (st == SSD_OK) st = check_map(a.sl, T);
    if (st != SSD_OK) return st;
    if (T > 0 && (!y || (nslots > 0 && !states))) return SSD_ERR_INVALID_ARG;
    const size_t need = ssd_diag_scan_workspace_bytes(nseq, T, E, N, G);
    if (workspace_bytes < need || (need && (!workspace || !aligned(workspace, 16)))) return SSD_ERR_INVALID_ARG;
    const ScanRanges r = scan_ranges(a, elem_bytes(dtype));
    const MapRanges m = map_ranges(a.sl, T);
    if (clash({r.y, span(states, (int64_t)nslots * E * N * 4), span(workspace, (int64_t)need), m.status},
              {r.u, r.dt, r.z, r.B, r.C, r.A, r.bias, r.D, m.cu, m.seq, m.slot, m.init}))
        return SSD_ERR_INVALID_ARG;
    if ((int64_t)nseq + T > kMaxRows) return SSD_ERR_UNSUPPORTED;
    if (T == 0 || nseq == 0) return SSD_OK;
    return from_cuda(launch_diag_scan(a, stream));
}

size_t ssd_diag_scan_bwd_workspace_bytes(int b, int L, int E, int N, int G)
{
    if (b <= 0 || L <= 0 || (int64_t)b * L > kMaxRows || E <= 0 || N <= 0 || N > 64 || G <= 0 || E % G) return 0;
    return diag_scan_bwd_workspace_bytes(b, L, E, N, G);
}

ssd_status_t ssd_diag_scan_bwd(const void* u, int64_t u_stride, const void* dt_raw, int64_t dt_stride, const void* z,
                               int64_t z_stride, const void* B, const void* C, int64_t bc_stride, const float* A,
                               const float* dt_bias, const float* D, const float* init_state, const void* dy,
                               const float* dfinal, void* du, void* ddt_raw, void* dz, void* dB, void* dC, float* dA,
                               float* dD, float* ddt_bias, float* dinit, int b, int L, int E, int N, int G,
                               ssd_dtype_t dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    if (b < 0 || L < 0) return SSD_ERR_INVALID_ARG;
    if ((int64_t)b * L > kMaxRows) return SSD_ERR_UNSUPPORTED;
    DiagArgs f{u, dt_raw, z, B, C, u_stride, dt_stride, z_stride, bc_stride, A, dt_bias, D, init_state, nullptr, nullptr,
               b, L, b * L, E, N, G, dtype == SSD_BF16, SlotArgs{}, workspace};
    const ssd_status_t st = check_scan(f, dtype);
    if (st != SSD_OK) return st;
    const bool tokens = f.rows > 0;
    if (!dA || !dD || !ddt_bias || (tokens && (!dy || !du || !ddt_raw || !dB || !dC || (z && !dz)))) return SSD_ERR_INVALID_ARG;
    const int e = elem_bytes(dtype);
    if (!all_aligned({dy, dfinal, du, ddt_raw, dz, dA, dinit, workspace}, 16) || !all_aligned({dB, dC}, e) ||
        !all_aligned({dD, ddt_bias}, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t need = ssd_diag_scan_bwd_workspace_bytes(b, L, E, N, G);
    if (workspace_bytes < need || (need && !workspace)) return SSD_ERR_INVALID_ARG;
    const ScanRanges r = scan_ranges(f, e);
    const int64_t io = (int64_t)f.rows * E * e, bc = (int64_t)f.rows * G * N * e, st_bytes = (int64_t)b * E * N * 4;
    if (clash({span(du, io), span(ddt_raw, io), span(dz, z ? io : 0), span(dB, bc), span(dC, bc), span(dA, (int64_t)E * N * 4),
               span(dD, (int64_t)E * 4), span(ddt_bias, (int64_t)E * 4), span(dinit, dinit ? st_bytes : 0), span(workspace, (int64_t)need)},
              {r.u, r.dt, r.z, r.B, r.C, r.A, r.bias, r.D, span(dy, io), span(init_state, init_state ? st_bytes : 0),
               span(dfinal, dfinal ? st_bytes : 0)}))
        return SSD_ERR_INVALID_ARG;
    if (!tokens) {
        cudaError_t err = cudaMemsetAsync(dA, 0, (size_t)E * N * 4, stream);
        if (err == cudaSuccess) err = cudaMemsetAsync(dD, 0, (size_t)E * 4, stream);
        if (err == cudaSuccess) err = cudaMemsetAsync(ddt_bias, 0, (size_t)E * 4, stream);
        if (err == cudaSuccess && dinit && b > 0)
            err = dfinal ? cudaMemcpyAsync(dinit, dfinal, (size_t)st_bytes, cudaMemcpyDeviceToDevice, stream)
                         : cudaMemsetAsync(dinit, 0, (size_t)st_bytes, stream);
        return from_cuda(err);
    }
    const DiagBwdArgs a{f, dy, dfinal, du, ddt_raw, dz, dB, dC, dA, dD, ddt_bias, dinit};
    return from_cuda(launch_diag_scan_bwd(a, stream));
}

ssd_status_t ssd_diag_state_update(float* states, const void* u, int64_t u_stride, const void* dt_raw,
                                   int64_t dt_stride, const void* z, int64_t z_stride, const void* B, const void* C,
                                   int64_t bc_stride, const float* A, const float* dt_bias, const float* D, void* y,
                                   const int32_t* cu_seqlens, const int32_t* seq_of, const int64_t* slot_of,
                                   const int32_t* init_slot, int nseq, int rows, int E, int N, int G,
                                   int block_tokens, int nslots, ssd_dtype_t dtype, int32_t* status,
                                   cudaStream_t stream)
{
    DiagArgs a{u, dt_raw, z, B, C, u_stride, dt_stride, z_stride, bc_stride, A, dt_bias, D, states, y, states,
               nseq, 0, rows, E, N, G, dtype == SSD_BF16,
               SlotArgs{cu_seqlens, seq_of, slot_of, init_slot, nseq, nslots, block_tokens, status}, nullptr};
    ssd_status_t st = check_scan(a, dtype);
    if (st != SSD_OK) return st;
    if (cu_seqlens || seq_of || slot_of || init_slot) {
        if ((st = check_map(a.sl, rows)) != SSD_OK) return st;
    } else if (nslots < rows) {
        return SSD_ERR_INVALID_ARG;
    }
    if (rows > 0 && (!y || (nslots > 0 && !states))) return SSD_ERR_INVALID_ARG;
    const ScanRanges r = scan_ranges(a, elem_bytes(dtype));
    const MapRanges m = map_ranges(a.sl, rows);
    if (clash({r.y, span(states, (int64_t)nslots * E * N * 4), m.status},
              {r.u, r.dt, r.z, r.B, r.C, r.A, r.bias, r.D, m.cu, m.seq, m.slot, m.init}))
        return SSD_ERR_INVALID_ARG;
    if (rows > kMaxRows) return SSD_ERR_UNSUPPORTED;
    if (rows == 0) return SSD_OK;
    return from_cuda(launch_diag_update(a, stream));
}

}  // extern "C"
