// diag.h -- internal launch interface of the diagonal scan's kernels (the
// public one is include/ssd_diag.h; diag_api.cu validates and calls these).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

struct StateMapArgs {
    const int32_t *lens, *ctx, *table, *free_list, *free_head;
    int n, max_blocks, nfree, T, block, nslots;
    int32_t *cu, *seq_of, *pos_of;
    int64_t* slot_of;
    int32_t *init_slot, *table_out, *free_head_out;
    int32_t* ws;   // [0]: the batch is refused; [64 + r]: request r's first entry in free_list
    int32_t* status;
};
constexpr int kMapWsHeader = 64;
constexpr int kMapMaxSlots = 1500000;
// Rows and requests of a call: row numbers are ints, and the kernels step up to
// a tile or a piece past the last row.
constexpr int64_t kMaxRows = 0x7fffffff - (1 << 16);
cudaError_t launch_state_map(const StateMapArgs& a, cudaStream_t s);

struct SlotArgs {
    const int32_t* cu = nullptr;
    const int32_t* seq_of = nullptr;
    const int64_t* slot_of = nullptr;
    const int32_t* init_slot = nullptr;
    int nseq = 0, nslots = 0, block = 1;
    int32_t* status = nullptr;
};

cudaError_t launch_conv1d_varlen(const void* x, int64_t xs, void* out, int64_t os, const float* w, const float* bias,
                                 void* cache, const SlotArgs& sl, int T, int E, int k, bool bf16, cudaStream_t s);

size_t conv1d_bwd_workspace_bytes(int b, int L, int E, int k);
cudaError_t launch_conv1d_bwd(const void* x, const float* w, const float* bias, const void* conv_state,
                              const void* dout, void* dx, float* dw, float* dbias, void* dconv_state, int b, int L,
                              int E, int k, bool bf16, void* ws, cudaStream_t s);

// Rows of one diagonal scan: a dense batch (sl.cu null: b sequences of L
// rows, states init/final per sequence) or packed sequences with slots
// (init = final = the pool).
struct DiagArgs {
    const void *u, *dt, *z, *B, *C;
    int64_t us, dts, zs, bcs;
    const float *A, *dt_bias, *D, *init;
    void* y;
    float* final_state;
    int nseq, L, rows, E, N, G;
    bool bf16;
    SlotArgs sl;
    void* ws;
    // for the backward pass (launch_diag_ckpt)
    const void* dy = nullptr;
    float *ckpt = nullptr, *gl = nullptr, *gsdt = nullptr;
    int bseg = 0;
    bool longest_first = false;   // packed: sequences are taken up by length
    bool bc_aligned = false;   // every 4 elements of a B or C row are aligned to their size
};
inline bool bc_aligned(const DiagArgs& a, size_t elem)
{
    return a.bcs % 4 == 0 && reinterpret_cast<uintptr_t>(a.B) % (4 * elem) == 0 && reinterpret_cast<uintptr_t>(a.C) % (4 * elem) == 0;
}
// Of packed sequences, whatever their lengths; and of dense ones.
size_t diag_scan_workspace_bytes(int nseq, int rows, int E, int N, int G);
size_t diag_scan_fwd_workspace_bytes(int b, int L, int E, int N, int G);
cudaError_t launch_diag_scan(const DiagArgs& a, cudaStream_t s);
cudaError_t launch_diag_update(const DiagArgs& a, cudaStream_t s);

// What the backward pass starts from.  The states before every kDiagCkpt-th
// row of each sequence, to a.ckpt [nseq][ckpts_of(L)][E][N].  Where it walks
// the rows in pieces of a.bseg < L (a multiple of 32): for each piece [nseq]
// [pieces] the part of the state gradient at its start that comes from its
// own rows, to a.gl [E][N], and the sum of its dt, to a.gsdt [E].  The walk is
// itself cut every diag_ckpt_rows(...) rows (L: not at all), with
// diag_cut_bytes(...) of workspace at a.ws.
constexpr int kDiagCkpt = 4;
#ifdef __CUDACC__
__host__ __device__
#endif
inline int64_t ckpts_of(int L) { return ((int64_t)L + kDiagCkpt - 1) / kDiagCkpt; }
int diag_ckpt_rows(int b, int L, int E, int N, int G, int bseg);
size_t diag_cut_bytes(int nseq, int64_t pieces, int E, int N);
cudaError_t launch_diag_ckpt(const DiagArgs& a, cudaStream_t s);

struct DiagBwdArgs {
    DiagArgs f;            // the forward call's inputs
    const void* dy;
    const float* dfinal;
    void *du, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *ddt_bias, *dinit;
};
size_t diag_scan_bwd_workspace_bytes(int b, int L, int E, int N, int G);
cudaError_t launch_diag_scan_bwd(const DiagBwdArgs& a, cudaStream_t s);

// lanes that share a channel, each with 4 states: the power of two that holds N
inline int diag_lanes(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

inline int sm_count()
{
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 148;   // no device: sizes are still asked for on hosts without one
    }
    return v;
}

}  // namespace ssd
