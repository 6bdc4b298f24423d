// diag.cuh -- device helpers of the diagonal selective scan's kernels.
#pragma once

#include "common.cuh"
#include "ssd.h"

namespace ssd {

constexpr float kLog2e = 1.4426950408889634f;

// A log2(e), the factor of dt in a decay's exponent.  Held to finite values: a
// state that forgets at once (A = -inf) would otherwise turn the rows that
// fill up a tile, whose dt is 0, into 0 * inf.
__device__ inline float decay_rate(float A)
{
    const float v = A * kLog2e;
    return v < -3.4028234e38f ? -3.4028234e38f : v;
}
__device__ inline float4 decay_rate(float4 A) { return make_float4(decay_rate(A.x), decay_rate(A.y), decay_rate(A.z), decay_rate(A.w)); }

// Packed fp32 pairs: one instruction, each half rounded as the scalar one.
__device__ inline float2 pk_fma(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ inline float2 pk_mul(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// 2^v on the special-function unit (2 ulp; results below 2^-126 become 0).
__device__ inline float ex2(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 1 / v on the special-function unit (1 ulp; 1 / inf is 0).
__device__ inline float rcp(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 1 / (1 + e^-v)
__device__ inline float sigmoid_f(float v) { return rcp(1.0f + ex2(v * -kLog2e)); }

// softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|) in [0, 1], with
// log1p(e) = 2 atanh(w), w = e / (2 + e) <= 1/3, by the series
// 2 w (1 + w^2/3 + ... + w^12/13): the first term left out is below 2e-8 of
// the sum, so the result is good to a few ulp at every v (an e of zero gives
// max(v, 0); NaN stays NaN).
__device__ inline float softplus_series(float v)
{
    const float e = expf(-fabsf(v));
    const float w = __fdividef(e, 2.0f + e);
    const float q = w * w;
    float p = fmaf(q, 1.0f / 13.0f, 1.0f / 11.0f);
    p = fmaf(q, p, 1.0f / 9.0f);
    p = fmaf(q, p, 1.0f / 7.0f);
    p = fmaf(q, p, 1.0f / 5.0f);
    p = fmaf(q, p, 1.0f / 3.0f);
    p = fmaf(q, p, 1.0f);
    return fmaxf(v, 0.0f) + (w + w) * p;
}

// The same on a pair, in packed arithmetic, with e = 2^(-|v| log2 e) from the
// hardware exponential (its argument's rounding adds |v| 2^-24 to e's
// relative error).
__device__ inline float2 softplus_pair(float2 v)
{
    const float2 e = make_float2(ex2(fabsf(v.x) * -kLog2e), ex2(fabsf(v.y) * -kLog2e));
    // (one reciprocal for both would let a NaN of one row into the other)
    const float2 w = pk_mul(e, make_float2(rcp(2.0f + e.x), rcp(2.0f + e.y)));
    const float2 q = pk_mul(w, w);
    auto both = [](float c) { return make_float2(c, c); };
    float2 p = pk_fma(q, both(1.0f / 13.0f), both(1.0f / 11.0f));
    p = pk_fma(q, p, both(1.0f / 9.0f));
    p = pk_fma(q, p, both(1.0f / 7.0f));
    p = pk_fma(q, p, both(1.0f / 5.0f));
    p = pk_fma(q, p, both(1.0f / 3.0f));
    p = pk_fma(q, p, both(1.0f));
    return pk_fma(pk_mul(w, both(2.0f)), p, make_float2(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)));
}

// d SiLU(v) / dv, given sigmoid(v)
__device__ inline float dsilu_f(float v, float sg) { return sg * fmaf(v, 1.0f - sg, 1.0f); }

// Sums of v[0 .. NV) over LANES lanes (STRIDE apart), each lane keeping a part:
// v[i] ends as the sum of value `first + i`, i < max(1, NV / LANES).
template <int NV, int LANES, int STRIDE>
__device__ inline void scatter_sum(float* v, int l, int& first)
{
    if constexpr (LANES > 1) {
        if constexpr (NV > 1) {
            const bool up = l & (LANES / 2);
#pragma unroll
            for (int i = 0; i < NV / 2; ++i) {
                const float keep = up ? v[NV / 2 + i] : v[i], send = up ? v[i] : v[NV / 2 + i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, LANES / 2 * STRIDE);
            }
            if (up) first += NV / 2;
            scatter_sum<NV / 2, LANES / 2, STRIDE>(v, l, first);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], LANES / 2 * STRIDE);
            scatter_sum<1, LANES / 2, STRIDE>(v, l, first);
        }
    }
}

// 8 adjacent elements as they lie in memory: 16 bytes (bf16) or 32 (f32).
template <typename T> struct Raw8 {
    uint4 q[sizeof(T) / 2];
    __device__ inline void zero()
    {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) q[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ inline void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) q[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ inline float get(int j) const { return io<T>::word_get(reinterpret_cast<const uint32_t*>(q), j); }
    __device__ static inline void store(T* p, const float (&v)[8])
    {
        if constexpr (sizeof(T) == 2) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
};

// 4 adjacent elements of any alignment; `vec`: they are aligned to their size.
template <typename T> __device__ inline void load4(const T* p, bool vec, float (&v)[4])
{
    if (vec) {
        if constexpr (sizeof(T) == 2) {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
            v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
            v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
        } else {
            const float4 q = __ldg(reinterpret_cast<const float4*>(p));
            v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ld_f(p + i);
    }
}

// A packed batch's requests and state slots (device pointers; see ssd_diag.h).
struct Slots {
    const int32_t* cu;         // [nseq + 1]
    const int32_t* seq_of;     // [T]
    const int64_t* slot_of;    // [T]
    const int32_t* init_slot;  // [nseq]
    int nseq, nslots, block;
    int32_t* status;
};

__device__ inline void flag_invalid(int32_t* status)
{
    if (status) atomicExch(reinterpret_cast<int*>(status), (int)SSD_ERR_INVALID_ARG);
}

// A flat place in the pool as slot and place in the block.  The 64-bit divide
// costs a hundred instructions; places below 2^32 take the 32-bit one.
__device__ inline void split_place(int64_t flat, int block, int64_t& slot, int& off)
{
    if ((uint64_t)flat >> 32) {
        slot = flat / block;
        off = (int)(flat - slot * block);
    } else {
        const uint32_t q = (uint32_t)flat / (uint32_t)block;
        slot = q;
        off = (int)((uint32_t)flat - q * (uint32_t)block);
    }
}

// The slot that a row's block lives in, or -1 (and the status word set) if
// the map names none.
__device__ inline int slot_at(const Slots& s, int64_t flat)
{
    int64_t slot;
    int off;
    split_place(flat, s.block, slot, off);   // a negative place is beyond any pool
    if (flat < 0 || slot >= s.nslots) {
        flag_invalid(s.status);
        return -1;
    }
    return (int)slot;
}

// The place in its block of a row (0 for a place the map does not name).
__device__ inline int block_offset(const Slots& s, int64_t flat)
{
    int64_t slot;
    int off;
    split_place(flat, s.block, slot, off);
    return flat < 0 ? 0 : off;
}

// One piece of one sequence: the rows t0 .. t1-1 of sequence r = [s0, s1).
// The pieces of a sequence are numbered first, next, next + 1, ..; idx is this
// one's.
struct Piece {
    int r, t0, t1, s0, s1;
    int64_t idx, first, next;
};

// Dense sequences of L rows are cut every seg rows: piece q is the
// (q % per)-th of sequence q / per.
__host__ __device__ inline int pieces_per(int L, int seg) { return (int)(((int64_t)L + seg - 1) / seg); }

__device__ inline bool find_piece_dense(int q, int L, int seg, Piece& p)
{
    const int per = pieces_per(L, seg);
    p.r = q / per;
    const int j = q - p.r * per;
    p.s0 = p.r * L;
    p.s1 = p.s0 + L;
    p.t0 = p.s0 + j * seg;
    p.t1 = j + 1 < per ? p.t0 + seg : p.s1;
    p.idx = q;
    p.first = (int64_t)p.r * per;
    p.next = p.first + 1;
    return true;
}

// Packed sequences are cut at the multiples of seg along the packed rows, so
// that each piece is found from its index alone: index q < nseq is sequence
// q's first piece, index nseq + m - 1 the piece that starts at row m * seg
// where that row lies inside a sequence.  A row at most `keep` rows behind its
// sequence's start begins no piece (the first piece runs on over it).
__device__ inline bool find_piece_packed(int q, const Slots& sl, int rows, int seg, int keep, Piece& p)
{
    auto bounds = [&](int r) {
        p.r = r;
        p.s0 = sl.cu[r];
        p.s1 = sl.cu[r + 1];
        if (p.s0 >= 0 && p.s1 >= p.s0 && p.s1 <= rows) return true;
        flag_invalid(sl.status);
        return false;
    };
    if (q < sl.nseq) {
        if (!bounds(q) || p.s1 == p.s0) return false;
        p.t0 = p.s0;
    } else {
        const int64_t at = (int64_t)(q - sl.nseq + 1) * seg;
        if (at >= rows) return false;
        const int r = sl.seq_of[at];
        if (r < 0) return false;       // behind the last sequence
        if (r >= sl.nseq) {
            flag_invalid(sl.status);
            return false;
        }
        if (!bounds(r)) return false;
        if (at < p.s0 || at >= p.s1) {
            flag_invalid(sl.status);
            return false;
        }
        if (at - p.s0 <= keep) return false;
        p.t0 = (int)at;
    }
    int64_t second = ((int64_t)p.s0 / seg + 1) * seg;   // where the sequence's second piece starts
    if (second - p.s0 <= keep) second += seg;           // (keep < seg)
    const int64_t cut = p.t0 == p.s0 ? second : (int64_t)p.t0 + seg;
    p.t1 = (int)(cut < p.s1 ? cut : p.s1);
    // the piece behind this one is found by its row's request: is it this one?
    if (cut < p.s1 && sl.seq_of[cut] != p.r) flag_invalid(sl.status);
    p.idx = q;
    p.first = p.r;
    p.next = sl.nseq + second / seg - 1;
    return true;
}

}  // namespace ssd
