// state_map.cu -- block tables and slot maps of a batch of requests, built on
// the device from the requests' lengths.
//
// Request r holds ctx[r] tokens in ceil(ctx / bs) blocks and brings lens[r]
// more, which open ceil((ctx + len) / bs) - ceil(ctx / bs) new ones.  Two
// prefix sums over the requests, of the new tokens and of the new blocks,
// give every row's request (by a binary search in cu_seqlens) and every new
// block's entry in the free list; row t at place p of request r then lies in
// block p / bs, at slot table[r][p / bs].
//
// The plan (prefix sums, every check, init slots) is one CTA's work: it reads
// a few numbers per request.  Which slots the batch writes is a bitmap over
// the pool in shared memory, so a slot written twice, or read by one request
// and written by another, is found in time linear in the requests.  The rows
// are then filled by a grid of CTAs that needs the plan only; a small batch
// is filled by the planning CTA itself, in the same launch, as the second
// launch would cost more than the fill.  In a graph, 24 requests of one token
// take 7.0 us; 700 requests and 262144 rows 11.7 (each kernel alone, from cold
// caches: 7 to plan, 10 to fill).
#include "diag.h"
#include "ssd.h"

namespace ssd {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kRowsPerThread = 4;

// Rows and table entries up to which the planning CTA fills by itself.
constexpr int kFillAlone = 4 * kPlanThreads;

__device__ inline int64_t blocks_of(int64_t tokens, int bs) { return (tokens + bs - 1) / bs; }

// The rows (4 per step) and the table entries of thread `tid` of `nthreads`.
__device__ inline void fill(const StateMapArgs& a, bool bad, int64_t tid, int64_t nthreads)
{
    const int32_t* base = a.ws + kMapWsHeader;
    const int used = bad ? 0 : a.cu[a.n];
    const int bs = a.block;
    for (int64_t t0 = tid * kRowsPerThread; t0 < a.T; t0 += nthreads * kRowsPerThread) {
        int seq[kRowsPerThread], pos[kRowsPerThread];
        int64_t slot[kRowsPerThread];
        int r = -1, next = 0;
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
            const int t = (int)t0 + i;
            seq[i] = pos[i] = -1;
            slot[i] = -1;
            if (t < used) {
                if (r < 0 || t >= next) {
                    // the last request whose rows begin at or before t
                    int lo = r < 0 ? 0 : r, hi = a.n;
                    while (hi - lo > 1) {
                        const int mid = (lo + hi) >> 1;
                        if (a.cu[mid] <= t) lo = mid;
                        else hi = mid;
                    }
                    r = lo;
                    next = a.cu[r + 1];
                }
                const int held = (int)blocks_of(a.ctx[r], bs);
                const int p = t - a.cu[r] + a.ctx[r];
                const int j = p / bs;
                const int sl = j < held ? a.table[(int64_t)r * a.max_blocks + j] : a.free_list[base[r] + j - held];
                seq[i] = r;
                pos[i] = p;
                slot[i] = (int64_t)sl * bs + (p - j * bs);
            }
        }
        if (t0 + kRowsPerThread <= a.T) {
            *reinterpret_cast<int4*>(a.seq_of + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
            *reinterpret_cast<int4*>(a.pos_of + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            longlong2* sp = reinterpret_cast<longlong2*>(a.slot_of + t0);
            sp[0] = make_longlong2(slot[0], slot[1]);
            sp[1] = make_longlong2(slot[2], slot[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kRowsPerThread; ++i)
                if (t0 + i < a.T) {
                    a.seq_of[t0 + i] = seq[i];
                    a.pos_of[t0 + i] = pos[i];
                    a.slot_of[t0 + i] = slot[i];
                }
        }
    }
    const int64_t entries = (int64_t)a.n * a.max_blocks;
    const bool in_place = a.table_out == a.table;
    for (int64_t e = tid; e < entries; e += nthreads) {
        const int r = (int)(e / a.max_blocks), j = (int)(e - (int64_t)r * a.max_blocks);
        bool fresh = false;
        int64_t held = 0;
        if (!bad) {
            held = blocks_of(a.ctx[r], a.block);
            fresh = j >= held && j < blocks_of((int64_t)a.ctx[r] + a.lens[r], a.block);
        }
        if (fresh) a.table_out[e] = a.free_list[base[r] + j - held];
        else if (!in_place) a.table_out[e] = a.table[e];
    }
}

template <bool ALONE>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const StateMapArgs a)
{
    extern __shared__ uint32_t written[];   // one bit per slot
    __shared__ long long warp_tok[32], warp_blk[32];
    __shared__ long long sum_tok, sum_blk;
    __shared__ int refused;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bs = a.block;
    int32_t* base = a.ws + kMapWsHeader;
    for (int i = tid; i < (a.nslots + 31) / 32; i += kPlanThreads) written[i] = 0;
    if (tid == 0) {
        sum_tok = sum_blk = 0;
        refused = 0;
    }
    const int head = *a.free_head;
    __syncthreads();
    auto mark = [&](int slot) {   // a second writer of a slot is refused
        if (slot < 0 || slot >= a.nslots || (atomicOr(&written[slot >> 5], 1u << (slot & 31)) >> (slot & 31) & 1u)) refused = 1;
    };
    for (int r0 = 0; r0 < a.n; r0 += kPlanThreads) {
        const int r = r0 + tid;
        long long tok = 0, blk = 0;
        if (r < a.n) {
            const long long len = a.lens[r], ctx = a.ctx[r];
            const long long held = blocks_of(ctx, bs), need = blocks_of(ctx + len, bs);
            if (len < 0 || ctx < 0 || ctx + len > 0x7fffffffLL || need > a.max_blocks) {
                refused = 1;
            } else {
                tok = len;
                blk = need - held;
                int slot = -1;
                if (ctx > 0) {
                    slot = a.table[(int64_t)r * a.max_blocks + (ctx - 1) / bs];
                    if (slot < 0 || slot >= a.nslots) refused = 1;
                    else if (len > 0 && ctx % bs) mark(slot);
                }
                a.init_slot[r] = slot;
            }
        }
        // exclusive prefix sums over the 1024 requests, on top of those before
        long long pt = tok, pb = blk;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long vt = __shfl_up_sync(0xffffffffu, pt, o), vb = __shfl_up_sync(0xffffffffu, pb, o);
            if (lane >= o) {
                pt += vt;
                pb += vb;
            }
        }
        if (lane == 31) {
            warp_tok[warp] = pt;
            warp_blk[warp] = pb;
        }
        __syncthreads();
        if (warp == 0) {
            long long wt = warp_tok[lane], wb = warp_blk[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long vt = __shfl_up_sync(0xffffffffu, wt, o), vb = __shfl_up_sync(0xffffffffu, wb, o);
                if (lane >= o) {
                    wt += vt;
                    wb += vb;
                }
            }
            warp_tok[lane] = wt;
            warp_blk[lane] = wb;
        }
        __syncthreads();
        const long long bt = sum_tok + (warp ? warp_tok[warp - 1] : 0) + pt - tok;
        const long long bb = sum_blk + (warp ? warp_blk[warp - 1] : 0) + pb - blk;
        if (r < a.n) {   // a sum beyond int32 is beyond T or the free list: refused below
            a.cu[r] = (int)bt;
            base[r] = (int)(head + bb);
        }
        __syncthreads();
        if (tid == 0) {
            sum_tok += warp_tok[31];
            sum_blk += warp_blk[31];
        }
        __syncthreads();
    }
    const long long tokens = sum_tok, fresh = sum_blk;
    if (tid == 0 && (tokens > a.T || head < 0 || head > a.nfree || fresh > a.nfree - head)) refused = 1;
    __syncthreads();
    if (!refused)
        for (int f = tid; f < (int)fresh; f += kPlanThreads) mark(a.free_list[head + f]);
    __syncthreads();
    // a state that is only read here (whole blocks, requests without new
    // tokens) must not be one that another request writes
    if (!refused)
        for (int r = tid; r < a.n; r += kPlanThreads) {
            const int slot = a.init_slot[r];
            if (slot >= 0 && (a.lens[r] == 0 || a.ctx[r] % bs == 0) && (written[slot >> 5] >> (slot & 31) & 1u)) refused = 1;
        }
    __syncthreads();
    const bool bad = refused != 0;
    if (bad)
        for (int r = tid; r < a.n; r += kPlanThreads) {
            a.cu[r] = 0;
            a.init_slot[r] = -1;
        }
    if (tid == 0) {
        a.cu[a.n] = bad ? 0 : (int)tokens;
        *a.free_head_out = bad ? head : head + (int)fresh;
        a.ws[0] = bad;
        if (bad) atomicExch(reinterpret_cast<int*>(a.status), (int)SSD_ERR_INVALID_ARG);
    }
    if constexpr (ALONE) {
        __syncthreads();
        fill(a, bad, tid, kPlanThreads);
    }
}

__global__ void __launch_bounds__(kFillThreads) fill_kernel(const StateMapArgs a)
{
    fill(a, a.ws[0] != 0, (int64_t)blockIdx.x * kFillThreads + threadIdx.x, (int64_t)gridDim.x * kFillThreads);
}

}  // namespace

cudaError_t launch_state_map(const StateMapArgs& a, cudaStream_t s)
{
    const size_t smem = (size_t)((a.nslots + 31) / 32) * 4;
    const int64_t entries = (int64_t)a.n * a.max_blocks;
    const bool alone = a.T <= kFillAlone && entries <= kFillAlone;
    const void* plan = alone ? (const void*)plan_kernel<true> : (const void*)plan_kernel<false>;
    if (smem > 40 * 1024) {
        // always the most that a call may need: another thread's smaller call
        // must not lower it between here and the launch
        const cudaError_t e = cudaFuncSetAttribute(plan, cudaFuncAttributeMaxDynamicSharedMemorySize, (kMapMaxSlots + 31) / 32 * 4);
        if (e != cudaSuccess) return e;
    }
    if (alone) plan_kernel<true><<<1, kPlanThreads, smem, s>>>(a);
    else plan_kernel<false><<<1, kPlanThreads, smem, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || alone) return e;
    const int64_t rows4 = ((int64_t)a.T + kRowsPerThread - 1) / kRowsPerThread;
    const int64_t threads = rows4 > entries ? rows4 : entries;
    const int64_t most = (int64_t)sm_count() * 8;
    int64_t ctas = (threads + kFillThreads - 1) / kFillThreads;
    if (ctas > most) ctas = most;
    fill_kernel<<<(unsigned)ctas, kFillThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ssd
