// conv1d_bwd.cu -- gradients of the causal depthwise conv1d + SiLU.
//
// With v_t = bias + sum_j w_j x_{t-k+1+j} and out = SiLU(v):
//   ds_t = dout_t SiLU'(v_t),   dx_t = sum_j w_j ds_{t+k-1-j},
//   dw_j = sum_t ds_t x_{t-k+1+j},   dbias = sum_t ds_t,
// x and dx taken over the cached columns too (times -k+1 .. -1).
//
// x and dout are read once, dx is written once.  A thread owns 4 adjacent
// channels and walks a tile of rows plus the k-1 behind them (whose ds it
// needs and recomputes), with the last k inputs and the last k ds in registers
// and a group of rows on the way while one is computed.  dw and dbias are
// summed in registers over the tile, written per tile, and summed over tiles
// by a second kernel in a fixed order: no atomics.
//
// Bound by latency: 8 x 2048 rows of 4608 bf16 channels are 576 CTAs, 14 warps
// an SM of the 16 that 128 registers allow, whose loads are what they wait for
// most (35% of a warp's time; issue is 44% busy, DRAM 50%, FMA 44%, special
// functions 37%).  104 us with the sum over tiles, 66% of the measured copy
// rate; 114 us with 128-row tiles, 125 with 512, 119 with groups of 2 rows, 139
// with 2 channels a thread.
#include "conv4.cuh"
#include "diag.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kCpt = 4;
constexpr int kTile = 256;
constexpr int kTileShort = 64;
constexpr int kGroup = 4;
constexpr int kRedCols = 32, kRedLanes = 8;

// Rows per tile: long tiles repeat less of their neighbours' work and start
// fewer CTAs, short ones fill the device where there is little to do.
inline int tile_rows(int b, int L, int E)
{
    const int64_t threads = (int64_t)b * (((int64_t)L + kTile - 1) / kTile) * (E / 4);
    return threads >= 148 * 256 ? kTile : kTileShort;
}
inline int tiles_of(int b, int L, int E)
{
    const int rows = tile_rows(b, L, E);
    return (int)(((int64_t)L + rows - 1) / rows);
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads)
conv1d_bwd_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ bias,
                  const T* __restrict__ conv_state, const T* __restrict__ dout, T* __restrict__ dx,
                  T* __restrict__ dconv_state, float* __restrict__ part, int L, int E, int rows)
{
    const int c0 = (blockIdx.y * kThreads + threadIdx.x) * kCpt;
    if (c0 >= E) return;
    const int ntile = (L + rows - 1) / rows;
    const int bi = blockIdx.x / ntile, tile = blockIdx.x - bi * ntile;
    const int t0 = tile * rows, t1 = min(L, t0 + rows);
    const int64_t row0 = (int64_t)bi * L;
    const T* xb = x + row0 * E + c0;
    const T* gb = dout + row0 * E + c0;
    T* dxb = dx + row0 * E + c0;

    // 4 channels as two fp32 pairs
    float2 wt[K][2], bs[2], dw[K][2], db[2];
    {
        float v[K][kCpt];
        load_taps<K>(w + (size_t)c0 * K, v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bs[h] = bias ? make_float2(bias[c0 + 2 * h], bias[c0 + 2 * h + 1]) : make_float2(0.0f, 0.0f);
            db[h] = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                wt[j][h] = make_float2(v[j][2 * h], v[j][2 * h + 1]);
                dw[j][h] = make_float2(0.0f, 0.0f);
            }
        }
    }
    // x[j]: the input j rows before this one; ds[j] likewise
    float2 xr[K][2], ds[K][2];
    auto pairs = [](const Row4<T>& q, float2 (&o)[2]) {
        float v[kCpt];
        q.get(v);
        o[0] = make_float2(v[0], v[1]);
        o[1] = make_float2(v[2], v[3]);
    };
#pragma unroll
    for (int j = 0; j < K; ++j) xr[j][0] = xr[j][1] = ds[j][0] = ds[j][1] = make_float2(0.0f, 0.0f);
    if (t0 > 0) {   // t0 >= rows >= K: the rows before are there
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            Row4<T> q;
            q.load(xb + (int64_t)(t0 - 1 - j) * E);
            pairs(q, xr[j]);
        }
    } else if (conv_state) {
        Cache4<T, K> old;
        old.load(conv_state + ((int64_t)bi * E + c0) * K);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            xr[j][0] = make_float2(old.get(0, K - 1 - j), old.get(1, K - 1 - j));
            xr[j][1] = make_float2(old.get(2, K - 1 - j), old.get(3, K - 1 - j));
        }
    }
    auto shift = [](float2 (&v)[K][2]) {
#pragma unroll
        for (int j = K - 1; j > 0; --j) {
            v[j][0] = v[j - 1][0];
            v[j][1] = v[j - 1][1];
        }
    };
    // Row t is taken in: ds_t and, where the tile owns it, its part of dw, db
    auto take = [&](const Row4<T>& qx, const Row4<T>& qg, bool own) {
        shift(xr);
        shift(ds);
        float2 g[2];
        pairs(qx, xr[0]);
        pairs(qg, g);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float2 v = bs[h];
#pragma unroll
            for (int j = 0; j < K; ++j) v = pk_fma(wt[j][h], xr[K - 1 - j][h], v);
            // SiLU'(v) = sg (1 + v (1 - sg)) = sg + (v sg) (1 - sg)
            const float2 sg = make_float2(sigmoid_f(v.x), sigmoid_f(v.y));
            const float2 d = pk_fma(pk_mul(v, sg), pk_fma(sg, make_float2(-1.0f, -1.0f), make_float2(1.0f, 1.0f)), sg);
            ds[0][h] = pk_mul(g[h], d);
            if (own) {
                db[h] = pk_fma(ds[0][h], make_float2(1.0f, 1.0f), db[h]);
#pragma unroll
                for (int j = 0; j < K; ++j) dw[j][h] = pk_fma(ds[0][h], xr[K - 1 - j][h], dw[j][h]);
            }
        }
    };
    // dx of the row K - 1 before the last one taken in
    auto give = [&](float (&o)[kCpt]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float2 v = pk_mul(wt[0][h], ds[0][h]);
#pragma unroll
            for (int j = 1; j < K; ++j) v = pk_fma(wt[j][h], ds[j][h], v);
            o[2 * h] = v.x;
            o[2 * h + 1] = v.y;
        }
    };
    auto next = [&](int t) {   // row t, or nothing behind the sequence
        if (t < L) {
            Row4<T> qx, qg;
            qx.load(xb + (int64_t)t * E);
            qg.load(gb + (int64_t)t * E);
            take(qx, qg, t < t1);
        } else {
            shift(ds);
            ds[0][0] = ds[0][1] = make_float2(0.0f, 0.0f);
        }
    };

    // the first K - 1 rows complete no row of this tile's; in a sequence's
    // first tile they complete the cached columns
    int t = t0;
    {
        Cache4<T, K> dcache;
        dcache.zero();
#pragma unroll
        for (int u = 0; u < K - 1; ++u, ++t) {
            next(t);
            float o[kCpt];
            give(o);
#pragma unroll
            for (int c = 0; c < kCpt; ++c) dcache.set(c, u + 1, o[c]);
        }
        if (t0 == 0 && dconv_state) dcache.store(dconv_state + ((int64_t)bi * E + c0) * K);
    }
    // whole groups, two sets of registers: one on its way while the other is used
    const T* xp = xb + (int64_t)t * E;
    const T* gp = gb + (int64_t)t * E;
    T* op = dxb + (int64_t)(t - (K - 1)) * E;
    struct Group {
        Row4<T> x[kGroup], g[kGroup];
    } ga, gbuf;
    auto fetch = [&](Group& q) {
#pragma unroll
        for (int u = 0; u < kGroup; ++u, xp += E, gp += E) {
            q.x[u].load(xp);
            q.g[u].load(gp);
        }
    };
    auto use = [&](const Group& q) {
#pragma unroll
        for (int u = 0; u < kGroup; ++u, op += E) {
            take(q.x[u], q.g[u], true);
            float o[kCpt];
            give(o);
            Row4<T>::store(op, o);
        }
    };
    int groups = (t1 - t) / kGroup;
    if (groups > 0) {
        t += groups * kGroup;
        fetch(ga);
        while (true) {
            if (groups > 1) fetch(gbuf);
            use(ga);
            if (--groups == 0) break;
            if (groups > 1) fetch(ga);
            use(gbuf);
            if (--groups == 0) break;
        }
    }
    for (; t < t1 + K - 1; ++t, op += E) {
        next(t);
        float o[kCpt];
        give(o);
        Row4<T>::store(op, o);
    }
    // [tile][K + 1][E]: taps, then the bias
    float* pr = part + (int64_t)blockIdx.x * (K + 1) * E + c0;
#pragma unroll
    for (int j = 0; j < K; ++j) *reinterpret_cast<float4*>(pr + (int64_t)j * E) = make_float4(dw[j][0].x, dw[j][0].y, dw[j][1].x, dw[j][1].y);
    *reinterpret_cast<float4*>(pr + (int64_t)K * E) = make_float4(db[0].x, db[0].y, db[1].x, db[1].y);
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
    const dim3 grid((unsigned)(b * tiles_of(b, L, E)), (unsigned)((E + per - 1) / per));
    conv1d_bwd_kernel<T, K><<<grid, kThreads, 0, s>>>(static_cast<const T*>(x), w, bias, static_cast<const T*>(conv_state),
                                                      static_cast<const T*>(dout), static_cast<T*>(dx),
                                                      static_cast<T*>(dconv_state), part, L, E, tile_rows(b, L, E));
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
    return (size_t)b * tiles_of(b, L, E) * (size_t)(k + 1) * E * 4;
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
        part, b * tiles_of(b, L, E), dw, dbias, E, k);
    return cudaGetLastError();
}

}  // namespace ssd
