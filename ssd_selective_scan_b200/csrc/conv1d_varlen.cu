// conv1d_varlen.cu -- causal depthwise conv1d + SiLU over packed requests,
// the rolling caches in slots (prompts of any lengths and single tokens).
//
// HBM-bound streaming, as the dense kernel: a thread owns 4 adjacent channels
// and walks a piece of one sequence, the k-1 previous inputs in registers.
// Pieces are cut at multiples of kPiece packed rows, so no CTA waits for a
// table of them; the piece that starts a sequence takes its left context
// from the init slot's cache and runs on where the next cut lies nearer than
// k-1 rows, so every other piece finds its left context in x.  Only a
// sequence's first piece therefore reads a cache, and it alone writes that
// same slot (where the sequence continues an unfinished block): a slot
// updated in place is read and written by one thread.  Slots of later blocks
// are written by the piece that holds the block's last row.
#include "conv4.cuh"
#include "diag.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kCpt = 4;      // channels per thread
constexpr int kPiece = 32;   // rows per piece
constexpr int kGroup = 8;    // rows loaded together

template <typename T, int K>
__global__ void __launch_bounds__(kThreads)
conv1d_varlen_kernel(const T* __restrict__ x, int64_t xs, T* __restrict__ out, int64_t os, const float* __restrict__ w,
                     const float* __restrict__ bias, T* cache, const Slots sl, int rows, int E)
{
    const int c0 = (blockIdx.y * kThreads + threadIdx.x) * kCpt;
    Piece p;
    if (!find_piece_packed(blockIdx.x, sl, rows, kPiece, K - 2, p) || c0 >= E) return;
    const T* xb = x + c0;
    const bool head = p.t0 == p.s0;
    const int init = head ? sl.init_slot[p.r] : -1;
    if (init >= sl.nslots) {
        flag_invalid(sl.status);
        return;
    }

    float wt[K][kCpt], bs[kCpt];
#pragma unroll
    for (int c = 0; c < kCpt; ++c) bs[c] = bias ? bias[c0 + c] : 0.0f;
    load_taps<K>(w + (size_t)c0 * K, wt);

    // hist[j]: the input K - 1 - j rows before the next one
    float hist[K][kCpt];
    Cache4<T, K> old;
    if (head) {
        if (init >= 0) old.load(cache + ((int64_t)init * E + c0) * K);
        else
#pragma unroll
            for (int i = 0; i < Cache4<T, K>::kWords; ++i) old.w[i] = 0;
#pragma unroll
        for (int j = 1; j < K; ++j)
#pragma unroll
            for (int c = 0; c < kCpt; ++c) hist[j - 1][c] = old.get(c, j);
    } else {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            Row4<T> q;
            q.load(xb + (int64_t)(p.t0 - (K - 1) + j) * xs);
            q.get(hist[j]);
        }
    }

    // A state ends at a row that is its block's last or the sequence's last;
    // the cache that goes to its slot is the K inputs up to there.  Rows
    // before the sequence come from the cache it started from.
    auto keep_state = [&](int t, int slot) {
        Cache4<T, K> now;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int at = t - (K - 1) + j;
            if (at >= p.s0) {
                Row4<T> q;
                float v[kCpt];
                q.load(xb + (int64_t)at * xs);
                q.get(v);
#pragma unroll
                for (int c = 0; c < kCpt; ++c) now.set(c, j, v[c]);
            } else {
                // only the head piece gets here: old column K + at - s0, a
                // register index that depends on at, so each is tried
                const int col = K + at - p.s0;
#pragma unroll
                for (int jj = 1; jj < K; ++jj)
                    if (jj == col)
#pragma unroll
                        for (int c = 0; c < kCpt; ++c) now.set(c, j, old.get(c, jj));
            }
        }
        now.store(cache + ((int64_t)slot * E + c0) * K);
    };

    // the first row in this piece at which a block ends
    const int64_t flat = sl.slot_of[p.t0];
    int64_t ends = (int64_t)p.t0 + sl.block - 1 - (flat < 0 ? 0 : flat % sl.block);
    if (flat < 0) flag_invalid(sl.status);

    if (head) {
        // the state in the block of the sequence's first row: this thread's to
        // write, wherever it ends, if it is the slot the sequence came from
        const int t = (int)(ends < p.s1 - 1 ? ends : p.s1 - 1);
        const int slot = slot_at(sl, sl.slot_of[t]);
        if (slot >= 0 && (slot == init || t < p.t1)) keep_state(t, slot);
    } else if (ends < p.t1 || p.t1 == p.s1) {
        const int t = (int)(ends < p.s1 - 1 ? ends : p.s1 - 1);
        const int slot = slot_at(sl, sl.slot_of[t]);
        // a block that began before this piece: the sequence's first block may
        // be the one it came from, which the head piece writes
        const int64_t begins = ends - sl.block + 1;
        if (slot >= 0 && !(begins <= p.s0 && slot == sl.init_slot[p.r])) keep_state(t, slot);
    }
    // blocks that begin inside this piece
    for (ends += 1; ends < p.t1; ends += sl.block) {
        const int64_t last = ends + sl.block - 1;
        const int64_t t = last < p.s1 - 1 ? last : p.s1 - 1;
        if (t >= p.t1) break;
        const int slot = slot_at(sl, sl.slot_of[t]);
        if (slot >= 0) keep_state((int)t, slot);
    }

    for (int tb = p.t0; tb < p.t1; tb += kGroup) {
        Row4<T> raw[kGroup];
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
            if (tb + u < p.t1) raw[u].load(xb + (int64_t)(tb + u) * xs);
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            if (tb + u < p.t1) {
                raw[u].get(hist[K - 1]);
                float2 a01 = make_float2(bs[0], bs[1]), a23 = make_float2(bs[2], bs[3]);
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    a01 = pk_fma(make_float2(wt[j][0], wt[j][1]), make_float2(hist[j][0], hist[j][1]), a01);
                    a23 = pk_fma(make_float2(wt[j][2], wt[j][3]), make_float2(hist[j][2], hist[j][3]), a23);
                }
                const float o[kCpt] = {silu_f(a01.x), silu_f(a01.y), silu_f(a23.x), silu_f(a23.y)};
                Row4<T>::store(out + (int64_t)(tb + u) * os + c0, o);
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
#pragma unroll
                    for (int c = 0; c < kCpt; ++c) hist[j][c] = hist[j + 1][c];
            }
        }
    }
}

template <typename T, int K>
cudaError_t launch_k(const void* x, int64_t xs, void* out, int64_t os, const float* w, const float* bias, void* cache,
                     const SlotArgs& a, int rows, int E, cudaStream_t s)
{
    const Slots sl{a.cu, a.seq_of, a.slot_of, a.init_slot, a.nseq, a.nslots, a.block, a.status};
    const int per = kThreads * kCpt;
    const dim3 grid((unsigned)(a.nseq + (rows - 1) / kPiece), (unsigned)((E + per - 1) / per));
    conv1d_varlen_kernel<T, K><<<grid, kThreads, 0, s>>>(static_cast<const T*>(x), xs, static_cast<T*>(out), os, w, bias,
                                                         static_cast<T*>(cache), sl, rows, E);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const void* x, int64_t xs, void* out, int64_t os, const float* w, const float* bias, void* cache,
                     const SlotArgs& a, int rows, int E, int k, cudaStream_t s)
{
    switch (k) {
        case 2: return launch_k<T, 2>(x, xs, out, os, w, bias, cache, a, rows, E, s);
        case 3: return launch_k<T, 3>(x, xs, out, os, w, bias, cache, a, rows, E, s);
        default: return launch_k<T, 4>(x, xs, out, os, w, bias, cache, a, rows, E, s);
    }
}

}  // namespace

cudaError_t launch_conv1d_varlen(const void* x, int64_t xs, void* out, int64_t os, const float* w, const float* bias,
                                 void* cache, const SlotArgs& a, int T, int E, int k, bool bf16, cudaStream_t s)
{
    return bf16 ? launch_t<__nv_bfloat16>(x, xs, out, os, w, bias, cache, a, T, E, k, s)
                : launch_t<float>(x, xs, out, os, w, bias, cache, a, T, E, k, s);
}

}  // namespace ssd
