// conv1d_bwd.cu -- gradients of the causal depthwise conv1d + SiLU.
//
// With v_t = bias + sum_j w_j x_{t-k+1+j} and out = SiLU(v):
//   ds_t = dout_t SiLU'(v_t),   dx_t = sum_j w_j ds_{t+k-1-j},
//   dw_j = sum_t ds_t x_{t-k+1+j},   dbias = sum_t ds_t,
// x and dx taken over the cached columns too (times -k+1 .. -1).
//
// HBM-bound streaming: x and dout are read once, dx is written once.  A
// thread owns 4 adjacent channels and walks kTile rows plus the k-1 behind
// them (whose ds it needs and recomputes: 5% of the reads, mostly from L2),
// with the last k inputs and the last k ds in registers.  dw and dbias are
// summed in registers over the tile (at most 64 terms), written per tile, and
// summed over tiles by a second kernel in a fixed order: no atomics.
#include "conv4.cuh"
#include "diag.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kCpt = 4;
constexpr int kTile = 64;
constexpr int kGroup = 4;
constexpr int kRedCols = 32, kRedLanes = 8;

__host__ __device__ inline int tiles_of(int L) { return (L + kTile - 1) / kTile; }

template <typename T, int K>
__global__ void __launch_bounds__(kThreads)
conv1d_bwd_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ bias,
                  const T* __restrict__ conv_state, const T* __restrict__ dout, T* __restrict__ dx,
                  T* __restrict__ dconv_state, float* __restrict__ part, int L, int E)
{
    const int c0 = (blockIdx.y * kThreads + threadIdx.x) * kCpt;
    if (c0 >= E) return;
    const int ntile = tiles_of(L);
    const int bi = blockIdx.x / ntile, tile = blockIdx.x - bi * ntile;
    const int t0 = tile * kTile, t1 = min(L, t0 + kTile);
    const int64_t row0 = (int64_t)bi * L;
    const T* xb = x + row0 * E + c0;
    const T* gb = dout + row0 * E + c0;
    T* dxb = dx + row0 * E + c0;

    float wt[K][kCpt], bs[kCpt], dw[K][kCpt], db[kCpt];
#pragma unroll
    for (int c = 0; c < kCpt; ++c) {
        bs[c] = bias ? bias[c0 + c] : 0.0f;
        db[c] = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            wt[j][c] = __ldg(w + (size_t)(c0 + c) * K + j);
            dw[j][c] = 0.0f;
        }
    }
    float hist[K][kCpt], ds[K][kCpt];   // ds[j]: ds of the row j before this one
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int c = 0; c < kCpt; ++c) hist[j][c] = ds[j][c] = 0.0f;
    if (t0 > 0) {   // t0 >= kTile >= K: the rows before are there
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            Row4<T> q;
            q.load(xb + (int64_t)(t0 - (K - 1) + j) * E);
            q.get(hist[j]);
        }
    } else if (conv_state) {
        Cache4<T, K> old;
        old.load(conv_state + ((int64_t)bi * E + c0) * K);
#pragma unroll
        for (int j = 1; j < K; ++j)
#pragma unroll
            for (int c = 0; c < kCpt; ++c) hist[j - 1][c] = old.get(c, j);
    }
    Cache4<T, K> dcache;
#pragma unroll
    for (int i = 0; i < Cache4<T, K>::kWords; ++i) dcache.w[i] = 0;

    for (int tb = t0; tb < t1 + K - 1; tb += kGroup) {
        Row4<T> rx[kGroup], rg[kGroup];
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
            if (tb + u < t1 + K - 1 && tb + u < L) {
                rx[u].load(xb + (int64_t)(tb + u) * E);
                rg[u].load(gb + (int64_t)(tb + u) * E);
            }
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            const int t = tb + u;
            if (t >= t1 + K - 1) break;
#pragma unroll
            for (int j = K - 1; j > 0; --j)
#pragma unroll
                for (int c = 0; c < kCpt; ++c) ds[j][c] = ds[j - 1][c];
            if (t < L) {
                float gv[kCpt];
                rx[u].get(hist[K - 1]);
                rg[u].get(gv);
#pragma unroll
                for (int c = 0; c < kCpt; ++c) {
                    float v = bs[c];
#pragma unroll
                    for (int j = 0; j < K; ++j) v = fmaf(wt[j][c], hist[j][c], v);
                    ds[0][c] = gv[c] * dsilu_f(v, sigmoid_f(v));
                    if (t < t1) {
                        db[c] += ds[0][c];
#pragma unroll
                        for (int j = 0; j < K; ++j) dw[j][c] = fmaf(ds[0][c], hist[j][c], dw[j][c]);
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < kCpt; ++c) ds[0][c] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int c = 0; c < kCpt; ++c) hist[j][c] = hist[j + 1][c];
            const int to = t - (K - 1);   // the row whose dx is now complete
            float o[kCpt];
#pragma unroll
            for (int c = 0; c < kCpt; ++c) {
                o[c] = 0.0f;
#pragma unroll
                for (int j = 0; j < K; ++j) o[c] = fmaf(wt[j][c], ds[j][c], o[c]);
            }
            if (to >= t0) {
                Row4<T>::store(dxb + (int64_t)to * E, o);
            } else if (to < 0) {          // a cached column: to + K, in 1 .. K-1
#pragma unroll
                for (int j = 1; j < K; ++j)
                    if (j == to + K)
#pragma unroll
                        for (int c = 0; c < kCpt; ++c) dcache.set(c, j, o[c]);
            }
        }
    }
    if (t0 == 0 && dconv_state) dcache.store(dconv_state + ((int64_t)bi * E + c0) * K);
    // [tile][K + 1][E]: taps, then the bias
    float* pr = part + (int64_t)blockIdx.x * (K + 1) * E + c0;
#pragma unroll
    for (int j = 0; j < K; ++j) *reinterpret_cast<float4*>(pr + (int64_t)j * E) = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
    *reinterpret_cast<float4*>(pr + (int64_t)K * E) = make_float4(db[0], db[1], db[2], db[3]);
}

// Sum over the tiles: 32 columns x 8 lanes of tiles per CTA, the lanes joined
// in shared memory in a fixed order.
__global__ void __launch_bounds__(kRedCols * kRedLanes)
conv1d_bwd_reduce_kernel(const float* __restrict__ part, int nparts, float* __restrict__ dw, float* __restrict__ dbias,
                         int E, int K)
{
    __shared__ float sums[kRedLanes][kRedCols];
    const int64_t cols = (int64_t)(K + 1) * E;
    const int64_t col = (int64_t)blockIdx.x * kRedCols + threadIdx.x;
    float acc = 0.0f;
    if (col < cols)
        for (int i = threadIdx.y; i < nparts; i += kRedLanes) acc += part[i * cols + col];
    sums[threadIdx.y][threadIdx.x] = acc;
    __syncthreads();
    if (threadIdx.y == 0 && col < cols) {
        acc = 0.0f;
#pragma unroll
        for (int i = 0; i < kRedLanes; ++i) acc += sums[i][threadIdx.x];
        const int j = (int)(col / E), e = (int)(col - (int64_t)j * E);
        if (j < K) dw[(int64_t)e * K + j] = acc;
        else if (dbias) dbias[e] = acc;
    }
}

template <typename T, int K>
void launch_k(const void* x, const float* w, const float* bias, const void* conv_state, const void* dout, void* dx,
              void* dconv_state, float* part, int b, int L, int E, cudaStream_t s)
{
    const int per = kThreads * kCpt;
    const dim3 grid((unsigned)(b * tiles_of(L)), (unsigned)((E + per - 1) / per));
    conv1d_bwd_kernel<T, K><<<grid, kThreads, 0, s>>>(static_cast<const T*>(x), w, bias, static_cast<const T*>(conv_state),
                                                      static_cast<const T*>(dout), static_cast<T*>(dx),
                                                      static_cast<T*>(dconv_state), part, L, E);
}

template <typename T>
void launch_t(const void* x, const float* w, const float* bias, const void* conv_state, const void* dout, void* dx,
              void* dconv_state, float* part, int b, int L, int E, int k, cudaStream_t s)
{
    if (k == 2) launch_k<T, 2>(x, w, bias, conv_state, dout, dx, dconv_state, part, b, L, E, s);
    else if (k == 3) launch_k<T, 3>(x, w, bias, conv_state, dout, dx, dconv_state, part, b, L, E, s);
    else launch_k<T, 4>(x, w, bias, conv_state, dout, dx, dconv_state, part, b, L, E, s);
}

}  // namespace

size_t conv1d_bwd_workspace_bytes(int b, int L, int E, int k)
{
    return (size_t)b * tiles_of(L) * (size_t)(k + 1) * E * 4;
}

cudaError_t launch_conv1d_bwd(const void* x, const float* w, const float* bias, const void* conv_state,
                              const void* dout, void* dx, float* dw, float* dbias, void* dconv_state, int b, int L,
                              int E, int k, bool bf16, void* ws, cudaStream_t s)
{
    float* part = static_cast<float*>(ws);
    if (bf16) launch_t<__nv_bfloat16>(x, w, bias, conv_state, dout, dx, dconv_state, part, b, L, E, k, s);
    else launch_t<float>(x, w, bias, conv_state, dout, dx, dconv_state, part, b, L, E, k, s);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t cols = (int64_t)(k + 1) * E;
    conv1d_bwd_reduce_kernel<<<(unsigned)((cols + kRedCols - 1) / kRedCols), dim3(kRedCols, kRedLanes), 0, s>>>(
        part, b * tiles_of(L), dw, dbias, E, k);
    return cudaGetLastError();
}

}  // namespace ssd
