// diag_scan.cu -- the diagonal selective scan, forward (dense batches, and
// packed requests with their states in slots).
//
//   h_t[e][n] = exp(dt_t[e] A[e][n]) h_{t-1}[e][n] + dt_t[e] u_t[e] B_t[n]
//   y_t[e]    = (sum_n h_t[e][n] C_t[n] + D[e] u_t[e]) SiLU(z_t[e])
//
// Every channel and state element decays at its own rate, so there is no
// matrix product to hand to the tensor cores: the work is one exponential and
// four FMAs per (token, channel, state).  What bounds it is the
// special-function unit (16 results per cycle and SM: N = 16 states cost a
// cycle per token and channel) and instruction issue, before HBM (8 bytes per
// token and channel).  8 x 2048 tokens of 2560 gated bf16 channels: 347 us,
// both at about 60% while an SM has work; 144 us for the exponentials alone.
//
// Layout.  A CTA covers CH channels of one group (diag_tile.cuh) and walks
// the tokens of a piece of a sequence in tiles of TT.  Two warps hold the
// states and run the recurrence; two more feed them, taking turns at the
// tiles: they copy u, dt_raw and z to shared memory ahead (cp.async), form dt
// = softplus(dt_raw + bias) and x = dt u once per (token, channel), lay them
// out with the tile's B and C rows, and finish the tile before: add D u to
// the sums over the states, gate, store 16-byte vectors.  Done by the same
// warps in turn these steps added their latencies to the recurrence's.  The
// sides meet at named barriers, a pair for each of the two tile buffers; a
// feeding warp has its next tile ready in registers when the buffer comes
// free.
//
// Rows lie in pairs, as the packed fp32 instructions take them: dt of rows 2i
// and 2i + 1 side by side, and so x, B and C.  exp, x B and the sum with C
// then work on both rows at once with no register copied; only the two steps
// of h itself are scalar.  y's sum over the states is finished 4 tokens at a
// time, each lane ending with two of them.
//
// Few rows.  A lane's tokens are a serial chain, and a narrow layer's single
// prompt has too few lanes to fill the device.  The rows are then cut into
// pieces (find_piece_dense, find_piece_packed): a first kernel walks every piece that has a successor
// from a zero state (a sequence's first piece from its initial state) and
// leaves its final state and the sum of its dt; a piece's true initial state
// is then the fold of those before it, exp(A sum dt) h + h_local, which the
// second kernel computes at its start before it walks the piece for y.  The
// exponentials are paid twice, so the rows are cut only where the lanes of
// one sequence leave the device idle (piece_rows).
#include <type_traits>

#include "diag_tile.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 2;                  // of each kind
constexpr int kThreads = 2 * 32 * kWarps;

// What a walk leaves: a piece's final state and sum of dt (in the workspace),
// y and the states, or what the backward pass starts from: the states every
// kDiagCkpt rows and, where it walks the rows in pieces, each piece's part of
// the state gradient at its start.
enum Mode { kLocal, kOutput, kCkpt, kCkptG };

template <typename T, int LPC, Mode MODE> struct Smem {
    using TL = DiagTile<LPC, kWarps>;
    static constexpr int NT = MODE == kCkptG ? 4 : MODE == kOutput ? 3 : 2;
    static constexpr int PAIRS = TL::TT / 2;
    float4 dx[2][PAIRS][TL::CH];                     // dt, dt', x, x' of two rows
    float4 B[2][PAIRS][LPC][2], C[2][PAIRS][LPC][2]; // b0, b0', b1, b1', b2, ..
    float2 p[MODE == kCkptG ? 2 : 1][MODE == kCkptG ? PAIRS : 1][TL::CH];   // dy SiLU(z)
    T raw[kWarps][3][NT][TL::TT][TL::CH];            // u, dt_raw, z, dy
};

// Packed sequences that a CTA ranks by length: one per thread, and only where
// they are long enough for a few hundred comparisons not to matter.
constexpr int kSortSeqs = kThreads;
constexpr int kSortRows = 128;   // rows per sequence

constexpr int kMeeting = 32 * (kWarps + 1);   // a feeding warp and the walking ones

// Named barriers of the two tile buffers: laid out, and walked.  The numbers
// are literals: a barrier number in a register makes the CTA hold all 16, and
// an SM then holds 4 CTAs at most.
template <int FIRST> __device__ inline void bar_sync(int buf)
{
    if (buf) asm volatile("bar.sync %0, %1;" ::"n"(FIRST + 1), "n"(kMeeting) : "memory");
    else asm volatile("bar.sync %0, %1;" ::"n"(FIRST), "n"(kMeeting) : "memory");
}
template <int FIRST> __device__ inline void bar_arrive(int buf)
{
    if (buf) asm volatile("bar.arrive %0, %1;" ::"n"(FIRST + 1), "n"(kMeeting) : "memory");
    else asm volatile("bar.arrive %0, %1;" ::"n"(FIRST), "n"(kMeeting) : "memory");
}
constexpr int kFull = 1, kDone = 3;


// Workspace of a cut scan: per piece its final state and sum of dt, and the
// initial state of every sequence (a piece that runs later may write the
// place it came from).
struct CutWs {
    float *h, *sdt, *h0;
};
__host__ __device__ inline CutWs cut_ws(void* ws, int64_t pieces, int E, int N)
{
    CutWs c;
    c.h = static_cast<float*>(ws);
    c.sdt = c.h + pieces * E * N;
    c.h0 = c.sdt + pieces * E;
    return c;
}
inline size_t cut_ws_bytes(int nseq, int64_t pieces, int E, int N) { return ((size_t)pieces * E * (N + 1) + (size_t)nseq * E * N) * 4; }

// CUT: the pieces' states are in the workspace.
template <typename T, int LPC, bool PACKED, Mode MODE, bool CUT>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 4) diag_scan_kernel(const DiagArgs a, int seg, int64_t pieces)
{
    using TL = DiagTile<LPC, kWarps>;
    constexpr bool OUT = MODE == kOutput, WITH_C = OUT || MODE == kCkptG;
    constexpr int TT = TL::TT, PAIRS = TT / 2, VPR = TL::VPR;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem<T, LPC, MODE>& sm = *reinterpret_cast<Smem<T, LPC, MODE>*>(smem_raw);

    const Slots sl{a.sl.cu, a.sl.seq_of, a.sl.slot_of, a.sl.init_slot, a.sl.nseq, a.sl.nslots, a.sl.block, a.sl.status};
    Piece p;
    const int ntiles = channel_tiles(a.E, a.G, TL::CH) * a.G;
    const int piece = (int)(blockIdx.x / ntiles);   // a piece's CTAs start together
    int which = piece;
    if constexpr (PACKED) {
        // longest sequences first, or the last ones to start are walked alone
        __shared__ int lens[kSortSeqs], chosen;
        if (a.longest_first && piece < a.nseq) {
            const int me = threadIdx.x;
            lens[me] = me < a.nseq ? sl.cu[me + 1] - sl.cu[me] : -1;
            __syncthreads();
            int rank = 0;
            for (int i = 0; i < a.nseq; ++i) rank += lens[i] > lens[me] || (lens[i] == lens[me] && i < me);
            if (me < a.nseq && rank == piece) chosen = me;
            __syncthreads();
            which = chosen;
        }
    }
    if (!(PACKED ? find_piece_packed(which, sl, a.rows, seg, seg - 1, p) : find_piece_dense(which, a.L, seg, p))) return;
    if (MODE == kLocal && p.t1 == p.s1) return;   // no successor

    const ChannelTile ct(a.E, a.G, TL::CH, blockIdx.x - piece * ntiles);
    const int e0 = ct.e0, e_end = ct.e_end;
    int init_at = -1;   // where the sequence's initial state is
    if constexpr (PACKED) {
        init_at = sl.init_slot[p.r];
        if (init_at >= sl.nslots) {
            flag_invalid(sl.status);
            return;
        }
    } else {
        init_at = a.init ? p.r : -1;
    }
    const int ntile = (p.t1 - p.t0 + TT - 1) / TT;
    // y's sums over the states, of the last 4 tiles
    __shared__ float2 ys[4][OUT ? PAIRS : 1][TL::CH];

    // The walking warps are the ones that need the special-function units, of
    // which each of the SM's four partitions has one; a warp runs on the
    // partition of its place on the SM modulo 4.  So which half of the CTA
    // walks goes by the CTA's place: neighbours take different halves.
    // (Wherever the places are, either half does the work.)
    __shared__ uint32_t place;
    if (threadIdx.x == 0) asm volatile("mov.u32 %0, %%warpid;" : "=r"(place));
    __syncthreads();
    const int me = (int)(threadIdx.x ^ ((place >> 2 & 1) * (32 * kWarps)));
    if (me >= 32 * kWarps) {
        // ---- the feeding warps, one to a buffer: rows 2 pr and 2 pr + 1, vector sv
        const int fl = me & 31, buf = (me >> 5) - kWarps;
        const int pr = fl / VPR, sv = fl % VPR;
        const int ev = e0 + 8 * sv;
        const bool copies = fl < PAIRS * VPR && ev < e_end;
        auto& raws = sm.raw[buf];
        const T* up = static_cast<const T*>(a.u) + ev;
        const T* dp = static_cast<const T*>(a.dt) + ev;
        const T* zp = static_cast<const T*>(a.z) + ev;
        const T* gp = static_cast<const T*>(a.dy) + ev;
        auto fetch = [&](int i) {        // tile i, on its way
            if (i < ntile && copies) {
                auto& raw = raws[(i >> 1) % 3];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int64_t row = p.t0 + i * TT + 2 * pr + k;
                    if (row >= p.t1) break;
                    cp_row8(&raw[0][2 * pr + k][8 * sv], up + row * a.us);
                    cp_row8(&raw[1][2 * pr + k][8 * sv], dp + row * a.dts);
                    if (WITH_C && a.z) cp_row8(&raw[2 * WITH_C][2 * pr + k][8 * sv], zp + row * a.zs);
                    if (MODE == kCkptG) cp_row8(&raw[MODE == kCkptG ? 3 : 0][2 * pr + k][8 * sv], gp + row * a.E);
                }
            }
            cp_commit();
        };
        // B and C: pair of rows bp, states 4 bq .. of this thread's items
        constexpr int ITEMS = (PAIRS * LPC + 31) / 32;
        const T* Bp = static_cast<const T*>(a.B) + (int64_t)ct.group * a.N;
        const T* Cp = static_cast<const T*>(a.C) + (int64_t)ct.group * a.N;
        const bool vec = a.bc_aligned;
        float bv[ITEMS][2][4], cv[ITEMS][2][4];
        auto fetch_bc = [&](int i) {
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int at = fl + 32 * k, bp = at / LPC, bq = at % LPC;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int64_t row = p.t0 + i * TT + 2 * bp + w;
                    const bool ok = at < PAIRS * LPC && row < p.t1 && 4 * bq < a.N;
#pragma unroll
                    for (int e = 0; e < 4; ++e) bv[k][w][e] = cv[k][w][e] = 0.0f;
                    if (ok) load4(Bp + row * a.bcs + 4 * bq, vec, bv[k][w]);
                    if (ok && WITH_C) load4(Cp + row * a.bcs + 4 * bq, vec, cv[k][w]);
                }
            }
        };
        // dt and x of tile i, in registers; rows behind the piece change nothing
        float2 dtv[8], xv[8], pv[MODE == kCkptG ? 8 : 1];
        auto form = [&](int i) {
            auto& raw = raws[(i >> 1) % 3];
            const int row = p.t0 + i * TT + 2 * pr;
            const bool ok0 = copies && row < p.t1, ok1 = copies && row + 1 < p.t1;
            if (!copies) return;
            const Raw8<T> u0 = smem_row8(&raw[0][2 * pr][8 * sv]), u1 = smem_row8(&raw[0][2 * pr + 1][8 * sv]);
            const Raw8<T> v0 = smem_row8(&raw[1][2 * pr][8 * sv]), v1 = smem_row8(&raw[1][2 * pr + 1][8 * sv]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float bias = a.dt_bias ? __ldg(a.dt_bias + ev + j) : 0.0f;
                const float2 dt = softplus_pair(make_float2(v0.get(j) + bias, v1.get(j) + bias));
                dtv[j] = make_float2(ok0 ? dt.x : 0.0f, ok1 ? dt.y : 0.0f);
                xv[j] = make_float2(ok0 ? dt.x * u0.get(j) : 0.0f, ok1 ? dt.y * u1.get(j) : 0.0f);
            }
            if constexpr (MODE == kCkptG) {
                const Raw8<T> z0 = smem_row8(&raw[2][2 * pr][8 * sv]), z1 = smem_row8(&raw[2][2 * pr + 1][8 * sv]);
                const Raw8<T> g0 = smem_row8(&raw[3][2 * pr][8 * sv]), g1 = smem_row8(&raw[3][2 * pr + 1][8 * sv]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float2 g = make_float2(g0.get(j), g1.get(j));
                    if (a.z) {
                        g.x *= z0.get(j) * sigmoid_f(z0.get(j));
                        g.y *= z1.get(j) * sigmoid_f(z1.get(j));
                    }
                    pv[j] = make_float2(ok0 ? g.x : 0.0f, ok1 ? g.y : 0.0f);
                }
            }
        };
        auto finish = [&](int i) {       // the outputs of tile i
            if constexpr (OUT) {
                if (!copies) return;
                auto& raw = raws[(i >> 1) % 3];
                float o[2][8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 y = ys[i & 3][pr][TL::col8(8 * sv + j, pr)];
                    o[0][j] = y.x;
                    o[1][j] = y.y;
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int64_t row = p.t0 + i * TT + 2 * pr + k;
                    if (row >= p.t1) break;
                    const Raw8<T> u = smem_row8(&raw[0][2 * pr + k][8 * sv]), z = smem_row8(&raw[2][2 * pr + k][8 * sv]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (a.D) o[k][j] = fmaf(__ldg(a.D + ev + j), u.get(j), o[k][j]);
                        if (a.z) {
                            const float zv = z.get(j);
                            o[k][j] *= zv * sigmoid_f(zv);
                        }
                    }
                    Raw8<T>::store(static_cast<T*>(a.y) + row * a.E + ev, o[k]);
                }
            }
        };
        fetch(buf);
        fetch(buf + 2);
        if (buf < ntile) {
            fetch_bc(buf);
            asm volatile("cp.async.wait_group 1;" ::: "memory");   // a thread reads back what it copied itself
            form(buf);
        }
        for (int i = buf; i < ntile; i += 2) {
            if (i >= 2) bar_sync<kDone>(buf);
            if (copies) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sm.dx[buf][pr][TL::col16(8 * sv + j, pr)] = make_float4(dtv[j].x, dtv[j].y, xv[j].x, xv[j].y);
                    if constexpr (MODE == kCkptG) sm.p[buf][pr][TL::col8(8 * sv + j, pr)] = pv[j];
                }
            }
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int at = fl + 32 * k, bp = at / LPC, bq = at % LPC;
                if (at < PAIRS * LPC) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        sm.B[buf][bp][bq][h] = make_float4(bv[k][0][2 * h], bv[k][1][2 * h], bv[k][0][2 * h + 1], bv[k][1][2 * h + 1]);
                        if (WITH_C) sm.C[buf][bp][bq][h] = make_float4(cv[k][0][2 * h], cv[k][1][2 * h], cv[k][0][2 * h + 1], cv[k][1][2 * h + 1]);
                    }
                }
            }
            bar_arrive<kFull>(buf);
            if (i >= 2) finish(i - 2);
            fetch(i + 4);
            if (i + 2 < ntile) {
                fetch_bc(i + 2);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                form(i + 2);
            }
        }
        const int last = ntile - 1 - ((ntile - 1 - buf) & 1);   // this warp's last tile
        if (last >= 0 && ntile > buf) {
            bar_sync<kDone>(buf);
            finish(last);
        }
        return;
    }

    // ---- the walking warps
    const int lane = me & 31, q = lane % LPC;
    const int64_t st_all = (int64_t)a.E * a.N;
    int cl[2];
    int64_t st[2];
    bool live[2];
    float A2[2][4], h[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        cl[j] = TL::channel(me >> 5, lane, j);
        live[j] = e0 + cl[j] < e_end && 4 * q < a.N;
        st[j] = (int64_t)(e0 + cl[j]) * a.N + 4 * q;
        for (int n = 0; n < 4; ++n) A2[j][n] = h[j][n] = 0.0f;
        if (live[j]) {
            const float4 v = decay_rate(__ldg(reinterpret_cast<const float4*>(a.A + st[j])));
            A2[j][0] = v.x; A2[j][1] = v.y; A2[j][2] = v.z; A2[j][3] = v.w;
        }
    }
    auto put4 = [](float* dst, const float (&v)[4]) { *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]); };
    const CutWs ws = cut_ws(a.ws, pieces, a.E, a.N);
    const bool head = p.t0 == p.s0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (!live[j]) continue;
        auto load_h = [&](const float* src) {
            const float4 v = *reinterpret_cast<const float4*>(src + st[j]);
            h[j][0] = v.x; h[j][1] = v.y; h[j][2] = v.z; h[j][3] = v.w;
        };
        if (!CUT || (head && (MODE == kLocal || p.t1 == p.s1))) {
            if (head && init_at >= 0) load_h(a.init + init_at * st_all);
            if (CUT && MODE == kLocal && head) put4(ws.h0 + p.r * st_all + st[j], h[j]);
        } else if (head) {
            load_h(ws.h0 + p.r * st_all);
        } else if (MODE != kLocal) {
            load_h(ws.h + p.first * st_all);
            for (int64_t i = p.next; i < p.idx; ++i) {
                const float sdt = ws.sdt[i * a.E + e0 + cl[j]];
                const float4 v = *reinterpret_cast<const float4*>(ws.h + i * st_all + st[j]);
                h[j][0] = fmaf(ex2(A2[j][0] * sdt), h[j][0], v.x);
                h[j][1] = fmaf(ex2(A2[j][1] * sdt), h[j][1], v.y);
                h[j][2] = fmaf(ex2(A2[j][2] * sdt), h[j][2], v.z);
                h[j][3] = fmaf(ex2(A2[j][3] * sdt), h[j][3], v.w);
            }
        }
    }

    // the next row at which a block ends inside the piece (packed)
    int64_t keep = 0x7fffffffffffLL;
    if (PACKED && OUT) {
        const int64_t flat = sl.slot_of[p.t0];
        if (flat >= 0) keep = (int64_t)p.t0 + sl.block - 1 - block_offset(sl, flat);
    }
    const int keep_end = min(p.t1, p.s1 - 1);   // the sequence's last state is written behind the walk
    float sdt[2] = {0.0f, 0.0f};
    // the backward pieces' part: P the product of the decays since the
    // piece's start, Gl = sum_t P_t C_t p_t
    float P[2][4], Gl[2][4];
    auto restart = [&] {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            sdt[j] = 0.0f;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                P[j][n] = 1.0f;
                Gl[j][n] = 0.0f;
            }
        }
    };
    restart();
    // kept states: every 4 rows, and pieces start at multiples of that
    static_assert(kDiagCkpt == 4, "a state is kept before each walk of 4 rows");
    [[maybe_unused]] float* kept = a.ckpt + ((int64_t)p.r * ckpts_of(a.L) + (p.t0 - p.s0) / kDiagCkpt) * st_all;
    [[maybe_unused]] int piece_end = MODE == kCkptG ? min(p.t0 + a.bseg, p.s1) : 0;

    for (int it = 0; it < ntile; ++it) {
        const int buf = it & 1, t = p.t0 + it * TT;
        const int groups = (min(TT, p.t1 - t) + 3) / 4;
        bar_sync<kFull>(buf);
        // 4 rows; KEEPS: a block may end in them
        auto walk4 = [&](int gr, auto keeps) {
            constexpr bool KEEPS = decltype(keeps)::value;
            if constexpr (MODE == kCkpt || MODE == kCkptG) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (live[j]) put4(kept + st[j], h[j]);
                kept += st_all;
            }
            [[maybe_unused]] float2 acc[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int pr = 2 * gr + i;
                const float4 bb[2] = {sm.B[buf][pr][q][0], sm.B[buf][pr][q][1]};
                float4 cc[2];
                if (WITH_C) cc[0] = sm.C[buf][pr][q][0], cc[1] = sm.C[buf][pr][q][1];
                float h0[2][4];   // the states after the pair's first row
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 d = sm.dx[buf][pr][TL::col16(cl[j], pr)];
                    const float2 xx = make_float2(d.z, d.w);
                    [[maybe_unused]] float2 pp;
                    if constexpr (MODE == kCkptG) pp = sm.p[buf][pr][TL::col8(cl[j], pr)];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float2 b2 = n & 1 ? make_float2(bb[n >> 1].z, bb[n >> 1].w) : make_float2(bb[n >> 1].x, bb[n >> 1].y);
                        // (scalar: a pair of A would have to be copied together)
                        const float a0 = ex2(A2[j][n] * d.x), a1 = ex2(A2[j][n] * d.y);
                        const float2 xb = pk_mul(xx, b2);
                        h0[j][n] = fmaf(a0, h[j][n], xb.x);
                        h[j][n] = fmaf(a1, h0[j][n], xb.y);
                        if constexpr (WITH_C) {
                            const float2 c2 = n & 1 ? make_float2(cc[n >> 1].z, cc[n >> 1].w) : make_float2(cc[n >> 1].x, cc[n >> 1].y);
                            if constexpr (OUT) {
                                const float2 hh = make_float2(h0[j][n], h[j][n]);
                                acc[j][i] = n ? pk_fma(hh, c2, acc[j][i]) : pk_mul(hh, c2);
                            } else {
                                const float P0 = P[j][n] * a0;
                                P[j][n] = P0 * a1;
                                const float2 cp = pk_mul(c2, pp);
                                Gl[j][n] = fmaf(P[j][n], cp.y, fmaf(P0, cp.x, Gl[j][n]));
                            }
                        }
                    }
                    if constexpr (!OUT) sdt[j] += d.x + d.y;
                }
                if constexpr (KEEPS) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int row = t + 2 * pr + k;
                        if (row == keep) {   // a block ends here: its state to its slot
                            if (row < keep_end) {
                                const int slot = slot_at(sl, sl.slot_of[row]);
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    if (slot >= 0 && live[j]) put4(a.final_state + slot * st_all + st[j], k ? h[j] : h0[j]);
                            }
                            keep += sl.block;
                        }
                    }
                }
            }
            if constexpr (OUT) {
                // slot 0's channel (diag_tile.cuh), then two of the rows
                float v[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    v[2 * i] = acc[0][i].x + __shfl_xor_sync(0xffffffffu, acc[1][i].x, LPC / 2);
                    v[2 * i + 1] = acc[0][i].y + __shfl_xor_sync(0xffffffffu, acc[1][i].y, LPC / 2);
                }
                if constexpr (LPC == 2) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) ys[it & 3][2 * gr + i][TL::col8(cl[0], 2 * gr + i)] = make_float2(v[2 * i], v[2 * i + 1]);
                } else {
                    const int up = q & 1;
                    float k0 = up ? v[2] : v[0], k1 = up ? v[3] : v[1];
                    k0 += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 1);
                    k1 += __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 1);
#pragma unroll
                    for (int o = 2; o < LPC / 2; o <<= 1) {
                        k0 += __shfl_xor_sync(0xffffffffu, k0, o);
                        k1 += __shfl_xor_sync(0xffffffffu, k1, o);
                    }
                    ys[it & 3][2 * gr + up][TL::col8(cl[0], 2 * gr + up)] = make_float2(k0, k1);
                }
            }
            if constexpr (MODE == kCkptG) {
                // a backward piece ends behind these rows, or with the sequence
                const int row = t + 4 * gr + 4;
                if (row >= piece_end) {
                    const int64_t i = (int64_t)p.r * pieces_per(a.L, a.bseg) + (piece_end - 1 - p.s0) / a.bseg;
                    piece_end = min(piece_end + a.bseg, p.s1);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (live[j]) {
                            put4(a.gl + i * st_all + st[j], Gl[j]);
                            if (q == 0) a.gsdt[i * a.E + e0 + cl[j]] = sdt[j];
                        }
                    restart();
                }
            }
        };
        if (groups == TT / 4 && !(PACKED && OUT && keep < t + TT)) {
#pragma unroll 2
            for (int gr = 0; gr < TT / 4; ++gr) walk4(gr, std::false_type{});
        } else {
#pragma unroll 1
            for (int gr = 0; gr < groups; ++gr) walk4(gr, std::integral_constant<bool, PACKED && OUT>{});
        }
        bar_arrive<kDone>(buf);
    }

#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if constexpr (OUT) {
            if (p.t1 == p.s1) {
                if constexpr (PACKED) {
                    const int slot = slot_at(sl, sl.slot_of[p.s1 - 1]);
                    if (slot >= 0 && live[j]) put4(a.final_state + slot * st_all + st[j], h[j]);
                } else if (live[j] && a.final_state) {
                    put4(a.final_state + p.r * st_all + st[j], h[j]);
                }
            }
        } else if (MODE == kLocal && live[j]) {
            put4(ws.h + p.idx * st_all + st[j], h[j]);
            if (q == 0) ws.sdt[p.idx * a.E + e0 + cl[j]] = sdt[j];
        }
    }
}

// Where rows are cut.  Nanoseconds a token for 1, 2, 3, 4 and 8 CTAs of 32
// channels on each SM (bf16, gated): 79, 93, 111, 132, 258; the first walk takes
// about two thirds of that.  One CTA to an SM gains from 4 pieces (79 L to
// 222 L / 4), two do not (93 L to 222 L / 2).
constexpr int kWarpsWanted = 148 * 8;   // walking warps of a cut scan
constexpr int kPiecesLeast = 3;
constexpr int kPieceLeast = 128;        // rows; a shorter piece costs more to join than it gains

// Rows per piece, or no cut (the rows' count): one sequence that had all the
// rows would get as many pieces as fill the device; sequences shorter than a
// piece stay whole (packed ones are cut into pieces of up to twice that).
int piece_rows(int rows, int E, int N, int G)
{
    const int ch = kWarps * 64 / tile_lanes(N);
    const int64_t pieces = kWarpsWanted / ((int64_t)channel_tiles(E, G, ch) * G * kWarps);
    if (pieces < kPiecesLeast) return rows;
    int64_t seg = (rows + pieces - 1) / pieces;
    seg = (seg + 31) / 32 * 32;
    if (seg < kPieceLeast) seg = kPieceLeast;
    return seg < rows ? (int)seg : rows;
}

int64_t piece_count(bool packed, int nseq, int L, int rows, int seg)
{
    return packed ? nseq + ((int64_t)rows - 1) / seg : (int64_t)nseq * pieces_per(L, seg);
}

template <typename T, int LPC, bool PACKED, Mode MODE, bool CUT>
cudaError_t launch_mode(const DiagArgs& a, int seg, int64_t pieces, cudaStream_t s)
{
    const int64_t grid = pieces * channel_tiles(a.E, a.G, DiagTile<LPC, kWarps>::CH) * a.G;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    constexpr int smem = (int)sizeof(Smem<T, LPC, MODE>);
    if (smem > 32 * 1024) {   // with the kernel's own arrays, beyond what needs no leave
        const cudaError_t e = cudaFuncSetAttribute((const void*)diag_scan_kernel<T, LPC, PACKED, MODE, CUT>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    diag_scan_kernel<T, LPC, PACKED, MODE, CUT><<<(unsigned)grid, kThreads, smem, s>>>(a, seg, pieces);
    return cudaGetLastError();
}

template <typename T, int LPC, bool PACKED, Mode MODE>
cudaError_t launch_lpc(const DiagArgs& a, int seg, cudaStream_t s)
{
    const bool cut = seg < (PACKED ? a.rows : a.L);
    if (!cut) return launch_mode<T, LPC, PACKED, MODE, false>(a, 0x7fffffff, a.nseq, s);
    const int64_t pieces = piece_count(PACKED, a.nseq, a.L, a.rows, seg);
    const cudaError_t e = launch_mode<T, LPC, PACKED, kLocal, true>(a, seg, pieces, s);
    return e != cudaSuccess ? e : launch_mode<T, LPC, PACKED, MODE, true>(a, seg, pieces, s);
}

template <typename T, bool PACKED, Mode MODE>
cudaError_t launch_t(const DiagArgs& args, int seg, cudaStream_t s)
{
    DiagArgs a = args;
    a.longest_first = PACKED && a.nseq > 1 && a.nseq <= kSortSeqs && a.rows / a.nseq >= kSortRows;
    a.bc_aligned = bc_aligned(a, sizeof(T));
    switch (tile_lanes(a.N)) {
        case 2: return launch_lpc<T, 2, PACKED, MODE>(a, seg, s);
        case 4: return launch_lpc<T, 4, PACKED, MODE>(a, seg, s);
        case 8: return launch_lpc<T, 8, PACKED, MODE>(a, seg, s);
        default: return launch_lpc<T, 16, PACKED, MODE>(a, seg, s);
    }
}

}  // namespace

size_t diag_scan_workspace_bytes(int nseq, int rows, int E, int N, int G)
{
    const int seg = piece_rows(rows, E, N, G);
    if (seg >= rows) return 0;
    // packed or dense: a dense batch has at most one short piece per sequence
    return cut_ws_bytes(nseq, nseq + ((int64_t)rows - 1) / seg + 1, E, N);
}

// (sequences no longer than a piece are launched whole: launch_lpc)
size_t diag_scan_fwd_workspace_bytes(int b, int L, int E, int N, int G)
{
    return piece_rows(b * L, E, N, G) < L ? diag_scan_workspace_bytes(b, b * L, E, N, G) : 0;
}

cudaError_t launch_diag_scan(const DiagArgs& a, cudaStream_t s)
{
    const int seg = piece_rows(a.rows, a.E, a.N, a.G);
    if (a.sl.cu) return a.bf16 ? launch_t<__nv_bfloat16, true, kOutput>(a, seg, s) : launch_t<float, true, kOutput>(a, seg, s);
    return a.bf16 ? launch_t<__nv_bfloat16, false, kOutput>(a, seg, s) : launch_t<float, false, kOutput>(a, seg, s);
}

cudaError_t launch_diag_ckpt(const DiagArgs& a, cudaStream_t s)
{
    const int seg = diag_ckpt_rows(a.nseq, a.L, a.E, a.N, a.G, a.bseg);
    if (a.bseg < a.L) return a.bf16 ? launch_t<__nv_bfloat16, false, kCkptG>(a, seg, s) : launch_t<float, false, kCkptG>(a, seg, s);
    return a.bf16 ? launch_t<__nv_bfloat16, false, kCkpt>(a, seg, s) : launch_t<float, false, kCkpt>(a, seg, s);
}

// Rows per piece of the walk that keeps states: as the forward scan's, to the
// nearest whole number of backward pieces.
int diag_ckpt_rows(int b, int L, int E, int N, int G, int bseg)
{
    const int64_t seg = piece_rows(b * L, E, N, G);
    const int64_t near = (seg + bseg / 2) / bseg * bseg;
    const int64_t whole = near > bseg ? near : bseg;
    return seg < L && whole < L ? (int)whole : L;
}

size_t diag_cut_bytes(int nseq, int64_t pieces, int E, int N) { return cut_ws_bytes(nseq, pieces, E, N); }

}  // namespace ssd
