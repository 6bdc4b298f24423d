// conv4.cuh -- 4 adjacent channels of a conv row or cache in one thread's
// registers (the packed conv and the conv's gradient).
#pragma once

#include "diag.cuh"

namespace ssd {

// 4 channels of one row.
template <typename T> struct Row4;
template <> struct Row4<float> {
    float4 q;
    __device__ void load(const float* p) { q = __ldcs(reinterpret_cast<const float4*>(p)); }
    __device__ void get(float (&v)[4]) const { v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w; }
    __device__ static void store(float* p, const float (&v)[4]) { *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]); }
};
template <> struct Row4<__nv_bfloat16> {
    uint2 q;
    __device__ void load(const __nv_bfloat16* p) { q = __ldcs(reinterpret_cast<const uint2*>(p)); }
    __device__ void get(float (&v)[4]) const
    {
        v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
        v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
    }
    __device__ static void store(__nv_bfloat16* p, const float (&v)[4])
    {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
};

// The cache of one thread's channels in one slot: 4 * K adjacent elements,
// moved as 16-byte vectors where they are a multiple of that, else 8-byte ones.
template <typename T, int K> struct Cache4 {
    static constexpr int kWords = 4 * K * (int)sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ void load(const T* p)
    {
        if constexpr (kWords % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 q = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 2; ++i) {
                const uint2 q = reinterpret_cast<const uint2*>(p)[i];
                w[2 * i] = q.x;
                w[2 * i + 1] = q.y;
            }
        }
    }
    __device__ void store(T* p) const
    {
        if constexpr (kWords % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 2; ++i) reinterpret_cast<uint2*>(p)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
        }
    }
    __device__ float get(int c, int j) const { return io<T>::word_get(w, c * K + j); }
    __device__ void set(int c, int j, float v) { io<T>::word_set(w, c * K + j, v); }
};

// The taps of a thread's 4 channels: 4 * K adjacent floats, K vectors.
template <int K>
__device__ inline void load_taps(const float* w, float (&wt)[K][4])
{
    float v[4 * K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(w) + i);
        v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < K; ++j) wt[j][c] = v[c * K + j];
}

}  // namespace ssd
