// diag_update.cu -- the diagonal recurrence for one token per request, by
// state slots (the decode step).
//
// HBM-bound: 8 bytes of state move per element (4 in, 4 out) for one
// exponential and four FMAs.  LPC lanes share a channel, 4 states (16 bytes)
// each, so a warp reads and writes 512 adjacent bytes of a state.  A CTA
// takes CH = 128 / LPC channels of kUpdRows rows: it looks the rows' slots up
// once, issues its state loads (kUpdRows x 16 bytes in flight per thread), and
// while those are on their way forms dt and x = dt u once per (row, channel)
// and lays them and the rows' B and C out in shared memory, so that the lanes
// of a channel do not each load and compute them again.  A, D and dt_bias are
// read once for the rows.  y's sums over a channel's lanes are exchanged for
// all rows at once, each lane ending with some of the rows.
//
// 256 rows of 8192 bf16 channels, 16 states, by slots: 55.8 us in a graph over
// several pools, 5.1 TB/s, 78% of the measured copy rate; 58 as single calls,
// 51 on one pool, part of which stays in L2.  (8 rows a CTA, 7 CTAs an SM: 60
// us; 16 rows: 73.)
#include "diag.cuh"
#include "diag.h"

namespace ssd {
namespace {

constexpr int kUpdThreads = 128;
constexpr int kUpdRows = 4;
constexpr int kUpdCtas = 12;   // per SM

template <typename T, int LPC, int ROWS>
__global__ void __launch_bounds__(kUpdThreads, kUpdCtas) diag_update_kernel(const DiagArgs a)
{
    constexpr int CH = kUpdThreads / LPC, NP = 4 * LPC;
    __shared__ float2 dx[ROWS][CH];                   // dt, x = dt u; y takes dt's place
    __shared__ float4 Bs[ROWS][LPC], Cs[ROWS][LPC];
    const int tid = threadIdx.x, q = tid % LPC, cl = tid / LPC;
    const int per_group = a.E / a.G, tiles = (per_group + CH - 1) / CH;
    const int g = blockIdx.y / tiles;
    const int e0 = g * per_group + (blockIdx.y - g * tiles) * CH;
    const int e_end = min(e0 + CH, (g + 1) * per_group);
    const int e = e0 + cl, n0 = q * 4;
    const bool live = e < e_end && n0 < a.N;
    const Slots sl{a.sl.cu, a.sl.seq_of, a.sl.slot_of, a.sl.init_slot, a.sl.nseq, a.sl.nslots, a.sl.block, a.sl.status};
    const int64_t slot_elems = (int64_t)a.E * a.N;
    const int64_t off = (int64_t)e * a.N + n0;
    const int i0 = blockIdx.x * ROWS;

    // rows -> slots; -1 to a row that is left out
    __shared__ int from[ROWS], to[ROWS];
    if (tid < ROWS) {
        const int i = i0 + tid;
        int f = -1, t = -1;
        if (i < a.rows) {
            if (!sl.cu) {
                f = t = i;
            } else {
                const int r = sl.seq_of[i];
                const int64_t flat = sl.slot_of[i];
                if (r >= 0) {
                    const bool sound = r < sl.nseq && sl.cu[r] == i && sl.cu[r + 1] == i + 1;
                    const int init = sound ? sl.init_slot[r] : 0;
                    if (!sound || init >= sl.nslots) {
                        flag_invalid(sl.status);
                    } else {
                        t = slot_at(sl, flat);
                        f = init;
                    }
                }
            }
        }
        from[tid] = f;
        to[tid] = t;
    }
    __syncthreads();
    float4 st[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        st[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (live && to[k] >= 0 && from[k] >= 0)
            st[k] = __ldcs(reinterpret_cast<const float4*>(a.init + from[k] * slot_elems + off));
    }

    // rows left out are staged too: their inputs exist (i < rows) and nothing of them is kept
    for (int k = tid; k < ROWS * CH; k += kUpdThreads) {
        const int row = k / CH, c = k % CH;
        const int64_t i = i0 + row;
        float2 v = make_float2(0.0f, 0.0f);
        if (i < a.rows && e0 + c < e_end) {
            v.x = softplus_series(ld_f(static_cast<const T*>(a.dt) + i * a.dts + e0 + c) + (a.dt_bias ? a.dt_bias[e0 + c] : 0.0f));
            v.y = v.x * ld_f(static_cast<const T*>(a.u) + i * a.us + e0 + c);
        }
        dx[row][c] = v;
    }
    for (int k = tid; k < ROWS * NP; k += kUpdThreads) {
        const int row = k / NP, n = k % NP;
        const int64_t i = i0 + row;
        const bool ok = i < a.rows && n < a.N;
        reinterpret_cast<float*>(Bs)[k] = ok ? ld_f(static_cast<const T*>(a.B) + i * a.bcs + g * a.N + n) : 0.0f;
        reinterpret_cast<float*>(Cs)[k] = ok ? ld_f(static_cast<const T*>(a.C) + i * a.bcs + g * a.N + n) : 0.0f;
    }
    float A2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (live) {
        const float4 v = decay_rate(__ldg(reinterpret_cast<const float4*>(a.A + off)));
        A2[0] = v.x; A2[1] = v.y; A2[2] = v.z; A2[3] = v.w;
    }
    __syncthreads();

    float acc[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const float2 d = dx[k][cl];
        const float4 b = Bs[k][q], c = Cs[k][q];
        float4 h = st[k];
        h.x = fmaf(ex2(d.x * A2[0]), h.x, d.y * b.x);
        h.y = fmaf(ex2(d.x * A2[1]), h.y, d.y * b.y);
        h.z = fmaf(ex2(d.x * A2[2]), h.z, d.y * b.z);
        h.w = fmaf(ex2(d.x * A2[3]), h.w, d.y * b.w);
        acc[k] = fmaf(h.x, c.x, fmaf(h.y, c.y, fmaf(h.z, c.z, h.w * c.w)));
        if (live && to[k] >= 0) __stcs(reinterpret_cast<float4*>(a.final_state + to[k] * slot_elems + off), h);
    }
    int at = 0;
    scatter_sum<ROWS, LPC, 1>(acc, q, at);
    constexpr int KEPT = LPC < ROWS ? ROWS / LPC : 1;
#pragma unroll
    for (int k = 0; k < KEPT; ++k) dx[at + k][cl].x = acc[k];
    __syncthreads();
    for (int k = tid; k < ROWS * CH; k += kUpdThreads) {
        const int row = k / CH, c = k % CH;
        const int64_t i = i0 + row;
        if (to[row] < 0 || e0 + c >= e_end) continue;
        float y = dx[row][c].x;
        if (a.D) y = fmaf(a.D[e0 + c], ld_f(static_cast<const T*>(a.u) + i * a.us + e0 + c), y);
        if (a.z) {
            const float zv = ld_f(static_cast<const T*>(a.z) + i * a.zs + e0 + c);
            y *= zv * sigmoid_f(zv);
        }
        static_cast<T*>(a.y)[i * a.E + e0 + c] = io<T>::from_f(y);
    }
}

template <typename T, int LPC>
cudaError_t launch_lpc(const DiagArgs& a, cudaStream_t s)
{
    constexpr int CH = kUpdThreads / LPC;
    const int tiles = (a.E / a.G + CH - 1) / CH * a.G;
    const dim3 grid((unsigned)((a.rows + kUpdRows - 1) / kUpdRows), (unsigned)tiles);
    diag_update_kernel<T, LPC, kUpdRows><<<grid, kUpdThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const DiagArgs& a, cudaStream_t s)
{
    switch (diag_lanes(a.N)) {
        case 1: return launch_lpc<T, 1>(a, s);
        case 2: return launch_lpc<T, 2>(a, s);
        case 4: return launch_lpc<T, 4>(a, s);
        case 8: return launch_lpc<T, 8>(a, s);
        default: return launch_lpc<T, 16>(a, s);
    }
}

}  // namespace

cudaError_t launch_diag_update(const DiagArgs& a, cudaStream_t s)
{
    return a.bf16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace ssd
