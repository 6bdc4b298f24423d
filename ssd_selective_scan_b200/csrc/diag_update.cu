// diag_update.cu -- the diagonal recurrence for one token per request, by
// state slots (the decode step).
//
// HBM-bound: 8 bytes of state move per element (4 in, 4 out) for one
// exponential and four FMAs.  LPC lanes share a channel, 4 states (16 bytes)
// each, so a warp reads and writes 512 adjacent bytes of a state.  A thread
// keeps its channel's A, D and dt_bias and walks kRows rows, all of whose
// state loads are issued before the first is used: the parameters are read
// once per kRows rows, and each thread has kRows x 16 bytes in flight.
#include "diag.cuh"
#include "diag.h"

namespace ssd {
namespace {

constexpr int kUpdThreads = 128;
constexpr int kUpdRows = 8;

template <typename T, int LPC, int ROWS>
__global__ void __launch_bounds__(kUpdThreads) diag_update_kernel(const DiagArgs a)
{
    constexpr int CH = kUpdThreads / LPC;
    const int q = threadIdx.x % LPC;
    const int e = blockIdx.y * CH + threadIdx.x / LPC;
    const int n0 = q * 4;
    const bool live = e < a.E && n0 < a.N;
    const int g = e < a.E ? e / (a.E / a.G) : 0;
    float A2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float Dv = 0.0f, bias = 0.0f;
    if (live) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(a.A + (size_t)e * a.N + n0));
        A2[0] = v.x * kLog2e; A2[1] = v.y * kLog2e; A2[2] = v.z * kLog2e; A2[3] = v.w * kLog2e;
    }
    if (e < a.E) {
        Dv = a.D ? a.D[e] : 0.0f;
        bias = a.dt_bias ? a.dt_bias[e] : 0.0f;
    }
    const Slots sl{a.sl.cu, a.sl.seq_of, a.sl.slot_of, a.sl.init_slot, a.sl.nseq, a.sl.nslots, a.sl.block, a.sl.status};
    const int64_t slot_elems = (int64_t)a.E * a.N;
    const int64_t off = (int64_t)e * a.N + n0;
    const int i0 = blockIdx.x * ROWS;

    // rows -> slots; -1 to a row that is left out
    int from[ROWS], to[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const int i = i0 + k;
        from[k] = to[k] = -1;
        if (i >= a.rows) continue;
        if (!sl.cu) {
            from[k] = to[k] = i;
            continue;
        }
        const int r = sl.seq_of[i];
        if (r < 0) continue;
        if (r >= sl.nseq || sl.cu[r] != i || sl.cu[r + 1] != i + 1) {
            flag_invalid(sl.status);
            continue;
        }
        const int init = sl.init_slot[r];
        if (init >= sl.nslots) {
            flag_invalid(sl.status);
            continue;
        }
        to[k] = slot_at(sl, sl.slot_of[i]);
        from[k] = init;
    }
    float4 st[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        st[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (live && to[k] >= 0 && from[k] >= 0)
            st[k] = __ldcs(reinterpret_cast<const float4*>(a.init + from[k] * slot_elems + off));
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        if (to[k] < 0) continue;
        const int64_t i = i0 + k;
        float4 h = st[k];
        float acc = 0.0f, uv = 0.0f;
        if (live) {
            uv = ld_f(static_cast<const T*>(a.u) + i * a.us + e);
            const float dt = softplus_series(ld_f(static_cast<const T*>(a.dt) + i * a.dts + e) + bias);
            const float x = dt * uv;
            const T* Bp = static_cast<const T*>(a.B) + i * a.bcs + g * a.N + n0;
            const T* Cp = static_cast<const T*>(a.C) + i * a.bcs + g * a.N + n0;
            h.x = fmaf(ex2(dt * A2[0]), h.x, x * ld_f(Bp + 0));
            h.y = fmaf(ex2(dt * A2[1]), h.y, x * ld_f(Bp + 1));
            h.z = fmaf(ex2(dt * A2[2]), h.z, x * ld_f(Bp + 2));
            h.w = fmaf(ex2(dt * A2[3]), h.w, x * ld_f(Bp + 3));
            acc = fmaf(h.x, ld_f(Cp + 0), fmaf(h.y, ld_f(Cp + 1), fmaf(h.z, ld_f(Cp + 2), h.w * ld_f(Cp + 3))));
            __stcs(reinterpret_cast<float4*>(a.final_state + to[k] * slot_elems + off), h);
        }
#pragma unroll
        for (int o = LPC / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (q == 0 && e < a.E) {
            float y = fmaf(Dv, uv, acc);
            if (a.z) {
                const float zv = ld_f(static_cast<const T*>(a.z) + i * a.zs + e);
                y *= zv * sigmoid_f(zv);
            }
            static_cast<T*>(a.y)[i * a.E + e] = io<T>::from_f(y);
        }
    }
}

template <typename T, int LPC>
cudaError_t launch_lpc(const DiagArgs& a, cudaStream_t s)
{
    constexpr int CH = kUpdThreads / LPC;
    const int tiles = (a.E + CH - 1) / CH;
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
