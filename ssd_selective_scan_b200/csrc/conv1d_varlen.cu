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
constexpr int kGroupFew = 2; // the same where long sequences are few: their registers would cost every CTA

// A thread's taps and bias.
template <int K> struct Taps {
    float w[K][kCpt], b[kCpt];
    __device__ void load(const float* wp, const float* bp, int c0)
    {
        load_taps<K>(wp + (size_t)c0 * K, w);
#pragma unroll
        for (int c = 0; c < kCpt; ++c) b[c] = bp ? bp[c0 + c] : 0.0f;
    }
    __device__ void apply(const float (&in)[K][kCpt], float (&o)[kCpt]) const
    {
        float2 a01 = make_float2(b[0], b[1]), a23 = make_float2(b[2], b[3]);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            a01 = pk_fma(make_float2(w[j][0], w[j][1]), make_float2(in[j][0], in[j][1]), a01);
            a23 = pk_fma(make_float2(w[j][2], w[j][3]), make_float2(in[j][2], in[j][3]), a23);
        }
        o[0] = a01.x * sigmoid_f(a01.x); o[1] = a01.y * sigmoid_f(a01.y);
        o[2] = a23.x * sigmoid_f(a23.x); o[3] = a23.y * sigmoid_f(a23.y);
    }
};

// The rows of one piece for the thread's 4 channels from c0, GROUP
// of them loaded together.
template <typename T, int K, int GROUP>
__device__ inline void walk_piece(const Piece& p, const T* x, int64_t xs, T* out, int64_t os, const Taps<K>& taps, T* cache,
                                  const Slots& sl, int E, int c0)
{
    const T* xb = x + c0;
    const bool head = p.t0 == p.s0;
    const int init = head ? sl.init_slot[p.r] : -1;
    if (init >= sl.nslots) {
        flag_invalid(sl.status);
        return;
    }

    // hist[j]: the input K - 1 - j rows before the next one
    float hist[K][kCpt];
    Cache4<T, K> old;
    if (head) {
        if (init >= 0) old.load(cache + ((int64_t)init * E + c0) * K);
        else old.zero();
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
    int64_t ends = (int64_t)p.t0 + sl.block - 1 - block_offset(sl, flat);
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

    for (int tb = p.t0; tb < p.t1; tb += GROUP) {
        Row4<T> raw[GROUP];
#pragma unroll
        for (int u = 0; u < GROUP; ++u)
            if (tb + u < p.t1) raw[u].load(xb + (int64_t)(tb + u) * xs);
#pragma unroll
        for (int u = 0; u < GROUP; ++u) {
            if (tb + u < p.t1) {
                raw[u].get(hist[K - 1]);
                float o[kCpt];
                taps.apply(hist, o);
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
__global__ void __launch_bounds__(kThreads)
conv1d_varlen_kernel(const T* __restrict__ x, int64_t xs, T* __restrict__ out, int64_t os, const float* __restrict__ w,
                     const float* __restrict__ bias, T* cache, const Slots sl, int rows, int E)
{
    const int c0 = (blockIdx.y * kThreads + threadIdx.x) * kCpt;
    Piece p;
    if (!find_piece_packed(blockIdx.x, sl, rows, kPiece, K - 2, p) || c0 >= E) return;
    Taps<K> taps;
    taps.load(w, bias, c0);
    walk_piece<T, K, kGroup>(p, x, xs, out, os, taps, cache, sl, E, c0);
}

// A piece among single tokens.  Out of line, with taps of its own, so that its
// registers are not every CTA's.
template <typename T, int K>
__device__ __noinline__ void walk_rare(int q, const T* x, int64_t xs, T* out, int64_t os, const float* w, const float* bias, T* cache,
                                       const Slots* slots, int rows, int E, int c0)
{
    const Slots sl = *slots;
    Piece p;
    if (!find_piece_packed(q, sl, rows, kPiece, K - 2, p)) return;
    Taps<K> taps;
    taps.load(w, bias, c0);
    walk_piece<T, K, kGroupFew>(p, x, xs, out, os, taps, cache, sl, E, c0);
}

// Batches of single tokens: a CTA takes SEQS sequences of its channels, so
// that their taps (64 bytes a thread, against 8 of x) are read once for all
// and their caches are on the way together.  Sequences of more tokens (a
// prompt among the single tokens) are walked in pieces: the first by the CTA
// that has the sequence, those behind by the CTAs in turn, one to each at most,
// as there are at most two rows to a sequence.
template <typename T, int K, int SEQS>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 6 : 4)
conv1d_tokens_kernel(const T* __restrict__ x, int64_t xs, T* __restrict__ out, int64_t os, const float* __restrict__ w,
                     const float* __restrict__ bias, T* cache, const __grid_constant__ Slots sl, int rows, int E)
{
    static_assert(2 * SEQS <= kPiece, "a CTA has one later piece at most");
    __shared__ int first[SEQS], count[SEQS], init[SEQS], slot[SEQS], later;
    if (threadIdx.x < SEQS) {
        const int r = blockIdx.x * SEQS + threadIdx.x;
        int n = 0, in = -1, s0 = 0;
        if (r < sl.nseq) {
            s0 = sl.cu[r];
            const int s1 = sl.cu[r + 1];
            in = sl.init_slot[r];
            if (s0 < 0 || s1 < s0 || s1 > rows || in >= sl.nslots) flag_invalid(sl.status);
            else n = s1 - s0;
        }
        first[threadIdx.x] = s0;
        count[threadIdx.x] = n;
        init[threadIdx.x] = in;
    } else if (threadIdx.x == 32) {   // does a piece begin at this CTA's row? (find_piece_packed checks the rest)
        const int64_t at = ((int64_t)blockIdx.x + 1) * kPiece;
        const int r = at < rows ? sl.seq_of[at] : -1;
        later = r >= 0 && !(r < sl.nseq && at - sl.cu[r] <= K - 2);
    }
    // what needs no lookup is on its way before the lookups are back, and the
    // slots to write are looked up while the inputs are on theirs
    const int c0 = (blockIdx.y * kThreads + threadIdx.x) * kCpt;
    const bool live = c0 < E;
    Taps<K> taps;
    if (live) taps.load(w, bias, c0);
    __syncthreads();
    Cache4<T, K> old[SEQS];
    Row4<T> in[SEQS];
#pragma unroll
    for (int i = 0; i < SEQS; ++i)
        if (live && count[i] == 1) {
            in[i].load(x + (int64_t)first[i] * xs + c0);
            if (init[i] >= 0) old[i].load(cache + ((int64_t)init[i] * E + c0) * K);
            else old[i].zero();
        }
    if (threadIdx.x < SEQS && count[threadIdx.x] == 1) slot[threadIdx.x] = slot_at(sl, sl.slot_of[first[threadIdx.x]]);
    __syncthreads();
    if (!live) return;
#pragma unroll
    for (int i = 0; i < SEQS; ++i) {
        if (count[i] == 1) {
            float v[K][kCpt], o[kCpt];
            Cache4<T, K> now;
            in[i].get(v[K - 1]);
#pragma unroll
            for (int j = 1; j < K; ++j)
#pragma unroll
                for (int c = 0; c < kCpt; ++c) v[j - 1][c] = old[i].get(c, j);
            taps.apply(v, o);
            Row4<T>::store(out + (int64_t)first[i] * os + c0, o);
#pragma unroll
            for (int j = 0; j < K; ++j)
#pragma unroll
                for (int c = 0; c < kCpt; ++c) now.set(c, j, v[j][c]);
            if (slot[i] >= 0) now.store(cache + ((int64_t)slot[i] * E + c0) * K);
        }
    }
#pragma unroll 1
    for (int i = 0; i <= SEQS; ++i) {
        if (i < SEQS ? count[i] <= 1 : !later) continue;
        walk_rare<T, K>(i < SEQS ? (int)blockIdx.x * SEQS + i : sl.nseq + (int)blockIdx.x, x, xs, out, os, w, bias, cache, &sl, rows, E, c0);
    }
}

template <typename T, int K>
cudaError_t launch_k(const void* x, int64_t xs, void* out, int64_t os, const float* w, const float* bias, void* cache,
                     const SlotArgs& a, int rows, int E, cudaStream_t s)
{
    const Slots sl{a.cu, a.seq_of, a.slot_of, a.init_slot, a.nseq, a.nslots, a.block, a.status};
    const int per = kThreads * kCpt;
    const unsigned cols = (unsigned)((E + per - 1) / per);
    if (rows <= 2 * (int64_t)a.nseq) {
        // 256 tokens of 8192 bf16 channels 14.7 us (2.9 TB/s), 512 24.8, 256 of 2560
        // 5.3, 16 of 4096 3.3; 4 sequences to a CTA, 4 CTAs an SM: 14.7, 26.3, 5.5,
        // 4.4; 8 and 3: 20.2, 30.6, 7.7, 6.7; 2 and 8 CTAs (spills) 15.2, 25.6, 5.7,
        // 3.7.  256 tokens of 8192 f32 channels 20.9 (24.3 with the rare walk in line).
        constexpr int SEQS = 2;
        conv1d_tokens_kernel<T, K, SEQS><<<dim3((unsigned)((a.nseq + SEQS - 1) / SEQS), cols), kThreads, 0, s>>>(
            static_cast<const T*>(x), xs, static_cast<T*>(out), os, w, bias, static_cast<T*>(cache), sl, rows, E);
        return cudaGetLastError();
    }
    const dim3 grid((unsigned)(a.nseq + (rows - 1) / kPiece), cols);
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
