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
// cycle per token and channel), before HBM (8 bytes per token and channel).
//
// Layout.  LPC lanes share a channel, 4 states each, so a CTA of 128 threads
// covers CH = 128 / LPC channels of one group.  It walks the tokens of a
// piece of a sequence in tiles of TT: u, dt_raw and z come in 16-byte vectors
// while the tile before is computed, dt = softplus(dt_raw + bias) and
// x = dt u are formed once per (token, channel) by the thread that loaded
// them and handed to the channel's lanes through shared memory, as are the
// tile's B and C rows.  The state stays in registers for the whole piece.
// y's sum over the states is finished 4 tokens at a time: each step of the
// exchange halves the tokens a lane keeps, so 4 lanes need 3 shuffles for 4
// tokens.  y goes back through shared memory to the loading threads, which
// add D u, gate and store 16-byte vectors.
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
#include "diag.cuh"
#include "diag.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;

template <int LPC> struct Tile {
    static constexpr int CH = kThreads / LPC;             // channels per CTA
    static constexpr int TT = LPC < 4 ? 8 * LPC : 32;     // tokens per tile
    static constexpr int NP = 4 * LPC;                    // states, padded
    static constexpr int VPR = CH / 8;                    // 8-element vectors per row
    static constexpr int NVEC = TT * VPR;                 // ... per tile: at most one per thread
    static constexpr int PAD = CH + 1;                    // float2 per row of the dt | x tile
    static_assert(NVEC <= kThreads, "one vector per thread");
};

template <int LPC> struct Smem {
    float2 dx[2][Tile<LPC>::TT * Tile<LPC>::PAD];   // dt, x = dt u; y takes dt's place
    float4 B[2][Tile<LPC>::TT * LPC];
    float4 C[2][Tile<LPC>::TT * LPC];
};

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

// What a walk leaves: a piece's final state and sum of dt (in the workspace),
// y and the states, or the states every kDiagCkpt rows.
enum Mode { kLocal, kOutput, kCkpt };

// CUT: the pieces' states are in the workspace.
template <typename T, int LPC, bool PACKED, Mode MODE, bool CUT>
__global__ void __launch_bounds__(kThreads) diag_scan_kernel(const DiagArgs a, int seg, int64_t pieces)
{
    constexpr bool FULL = MODE == kOutput;
    using TL = Tile<LPC>;
    constexpr int CH = TL::CH, TT = TL::TT, VPR = TL::VPR, PAD = TL::PAD;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem<LPC>& sm = *reinterpret_cast<Smem<LPC>*>(smem_raw);

    const Slots sl{a.sl.cu, a.sl.seq_of, a.sl.slot_of, a.sl.init_slot, a.sl.nseq, a.sl.nslots, a.sl.block, a.sl.status};
    Piece p;
    if (!(PACKED ? find_piece_packed(blockIdx.x, sl, a.rows, seg, 0, p) : find_piece_dense(blockIdx.x, a.L, seg, p))) return;
    if (MODE == kLocal && p.t1 == p.s1) return;   // no successor

    const int tid = threadIdx.x;
    const int q = tid % LPC, cl = tid / LPC;
    const int per_group = a.E / a.G, tiles = (per_group + CH - 1) / CH;
    const int g = blockIdx.y / tiles;
    const int e0 = g * per_group + (blockIdx.y - g * tiles) * CH;     // the CTA's first channel
    const int e_end = min(e0 + CH, (g + 1) * per_group);
    const int e = e0 + cl, n0 = 4 * q;
    const bool live = e < e_end && n0 < a.N;
    const int64_t st = (int64_t)e * a.N + n0;
    const int64_t st_all = (int64_t)a.E * a.N;

    float A2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (live) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(a.A + st));
        A2[0] = v.x * kLog2e; A2[1] = v.y * kLog2e; A2[2] = v.z * kLog2e; A2[3] = v.w * kLog2e;
    }

    // the piece's initial state
    int init_at = -1;
    if constexpr (PACKED) {
        init_at = sl.init_slot[p.r];
        if (init_at >= sl.nslots) {
            flag_invalid(sl.status);
            return;
        }
    } else {
        init_at = a.init ? p.r : -1;
    }
    float h[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    auto load_h = [&](const float* src) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
    };
    auto store_h = [&](float* dst) { *reinterpret_cast<float4*>(dst) = make_float4(h[0], h[1], h[2], h[3]); };
    const CutWs ws = cut_ws(a.ws, pieces, a.E, a.N);
    const bool head = p.t0 == p.s0;
    if (live) {
        if (!CUT || (head && (MODE == kLocal || p.t1 == p.s1))) {
            if (head && init_at >= 0) load_h(a.init + init_at * st_all + st);
            if (CUT && MODE == kLocal && head) store_h(ws.h0 + p.r * st_all + st);
        } else if (head) {
            load_h(ws.h0 + p.r * st_all + st);
        } else if (MODE != kLocal) {
            load_h(ws.h + p.first * st_all + st);
            for (int64_t i = p.next; i < p.idx; ++i) {
                const float sdt = ws.sdt[i * a.E + e];
                const float4 v = *reinterpret_cast<const float4*>(ws.h + i * st_all + st);
                h[0] = fmaf(ex2(A2[0] * sdt), h[0], v.x);
                h[1] = fmaf(ex2(A2[1] * sdt), h[1], v.y);
                h[2] = fmaf(ex2(A2[2] * sdt), h[2], v.z);
                h[3] = fmaf(ex2(A2[3] * sdt), h[3], v.w);
            }
        }
    }

    // staging: vector sv of row sr of each tile
    const int sr = tid / VPR, sv = tid % VPR;
    const bool stages = tid < TL::NVEC && e0 + 8 * sv < e_end;
    float Dv[8], bias[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        Dv[j] = FULL && stages && a.D ? a.D[e0 + 8 * sv + j] : 0.0f;
        bias[j] = stages && a.dt_bias ? a.dt_bias[e0 + 8 * sv + j] : 0.0f;
    }
    const T* up = static_cast<const T*>(a.u) + e0 + 8 * sv;
    const T* dp = static_cast<const T*>(a.dt) + e0 + 8 * sv;
    const T* zp = static_cast<const T*>(a.z) + e0 + 8 * sv;
    T* yp = static_cast<T*>(a.y) + e0 + 8 * sv;
    const T* Bp = static_cast<const T*>(a.B) + (int64_t)g * a.N;
    const T* Cp = static_cast<const T*>(a.C) + (int64_t)g * a.N;

    Raw8<T> u_now, z_now, u_next, z_next, dt_next;
    constexpr int NBC = (TT * TL::NP + kThreads - 1) / kThreads;   // B (and C) elements per thread and tile
    float b_next[NBC], c_next[NBC];
    auto fetch = [&](int t) {   // the tile that starts at row t: into registers
        u_next.zero();
        z_next.zero();
        if (stages && t + sr < p.t1) {
            u_next.load(up + (int64_t)(t + sr) * a.us);
            dt_next.load(dp + (int64_t)(t + sr) * a.dts);
            if (FULL && a.z) z_next.load(zp + (int64_t)(t + sr) * a.zs);
        }
#pragma unroll
        for (int i = 0; i < NBC; ++i) {
            const int k = tid + i * kThreads;
            const int row = k / TL::NP, n = k % TL::NP;
            const bool ok = k < TT * TL::NP && t + row < p.t1 && n < a.N;
            b_next[i] = ok ? ld_f(Bp + (int64_t)(t + row) * a.bcs + n) : 0.0f;
            if (FULL) c_next[i] = ok ? ld_f(Cp + (int64_t)(t + row) * a.bcs + n) : 0.0f;
        }
    };
    auto stage = [&](int t, int buf) {   // registers to shared memory; rows behind the piece change nothing
        if (tid < TL::NVEC) {
            const bool ok = stages && t + sr < p.t1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float dt = ok ? softplus_series(dt_next.get(j) + bias[j]) : 0.0f;
                sm.dx[buf][sr * PAD + 8 * sv + j] = make_float2(dt, ok ? dt * u_next.get(j) : 0.0f);
            }
        }
#pragma unroll
        for (int i = 0; i < NBC; ++i) {
            const int k = tid + i * kThreads;
            if (k < TT * TL::NP) {
                reinterpret_cast<float*>(sm.B[buf])[k] = b_next[i];
                if (FULL) reinterpret_cast<float*>(sm.C[buf])[k] = c_next[i];
            }
        }
    };

    // the next row at which a block ends inside the piece (packed)
    int64_t keep = 0x7fffffffffffLL;
    if (PACKED && FULL) {
        const int64_t flat = sl.slot_of[p.t0];
        if (flat >= 0) keep = (int64_t)p.t0 + sl.block - 1 - flat % sl.block;
    }
    const int keep_end = min(p.t1, p.s1 - 1);   // the sequence's last state is written behind the walk
    float sdt = 0.0f;

    fetch(p.t0);
    stage(p.t0, 0);
    u_now = u_next;
    z_now = z_next;
    __syncthreads();
    int buf = 0;
    for (int t = p.t0; t < p.t1; t += TT, buf ^= 1) {
        const bool more = t + TT < p.t1;
        if (more) fetch(t + TT);

        float2* dx = sm.dx[buf];
        const int groups = (min(TT, p.t1 - t) + 3) / 4;
        for (int gr = 0; gr < groups; ++gr) {
            if constexpr (MODE == kCkpt) {
                const int row = t + 4 * gr - p.s0;   // pieces start at multiples of kDiagCkpt
                if (row % kDiagCkpt == 0 && live)
                    store_h(a.ckpt + ((int64_t)p.r * ckpts_of(a.L) + row / kDiagCkpt) * st_all + st);
            }
            float acc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 4 * gr + i;
                const float2 d = dx[row * PAD + cl];
                const float4 b4 = sm.B[buf][row * LPC + q];
                const float2 dd = make_float2(d.x, d.x), xx = make_float2(d.y, d.y);
                const float2 e01 = pk_mul(make_float2(A2[0], A2[1]), dd), e23 = pk_mul(make_float2(A2[2], A2[3]), dd);
                const float2 x01 = pk_mul(make_float2(b4.x, b4.y), xx), x23 = pk_mul(make_float2(b4.z, b4.w), xx);
                const float2 h01 = pk_fma(make_float2(ex2(e01.x), ex2(e01.y)), make_float2(h[0], h[1]), x01);
                const float2 h23 = pk_fma(make_float2(ex2(e23.x), ex2(e23.y)), make_float2(h[2], h[3]), x23);
                h[0] = h01.x; h[1] = h01.y; h[2] = h23.x; h[3] = h23.y;
                if constexpr (FULL) {
                    const float4 c4 = sm.C[buf][row * LPC + q];
                    const float2 y2 = pk_fma(h01, make_float2(c4.x, c4.y), pk_mul(h23, make_float2(c4.z, c4.w)));
                    acc[i] = y2.x + y2.y;
                    if (PACKED && t + row == keep) {
                        // a block ends here: its state to its slot
                        if (t + row < keep_end) {
                            const int slot = slot_at(sl, sl.slot_of[t + row]);
                            if (slot >= 0 && live) store_h(a.final_state + slot * st_all + st);
                        }
                        keep += sl.block;
                    }
                } else if (MODE == kLocal) {
                    sdt += d.x;
                }
            }
            if constexpr (FULL) {
                // the channel's lanes join their sums; lane q & 3 ends with token q & 3
                if constexpr (LPC >= 4) {
                    const bool hi = q & 2, odd = q & 1;
                    float k0 = hi ? acc[2] : acc[0], k1 = hi ? acc[3] : acc[1];
                    const float s0 = hi ? acc[0] : acc[2], s1 = hi ? acc[1] : acc[3];
                    k0 += __shfl_xor_sync(0xffffffffu, s0, 2);
                    k1 += __shfl_xor_sync(0xffffffffu, s1, 2);
                    float k = odd ? k1 : k0;
                    k += __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 1);
#pragma unroll
                    for (int o = 4; o < LPC; o <<= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
                    if (LPC == 4 || q < 4) dx[(4 * gr + (q & 3)) * PAD + cl].x = k;
                } else if constexpr (LPC == 2) {
                    const bool odd = q & 1;
                    float k0 = odd ? acc[2] : acc[0], k1 = odd ? acc[3] : acc[1];
                    k0 += __shfl_xor_sync(0xffffffffu, odd ? acc[0] : acc[2], 1);
                    k1 += __shfl_xor_sync(0xffffffffu, odd ? acc[1] : acc[3], 1);
                    dx[(4 * gr + 2 * q) * PAD + cl].x = k0;
                    dx[(4 * gr + 2 * q + 1) * PAD + cl].x = k1;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) dx[(4 * gr + i) * PAD + cl].x = acc[i];
                }
            }
        }
        // the other buffer was last read before the barrier of the tile before
        // (its y by this thread alone, at the places it now writes)
        if (more) stage(t + TT, buf ^ 1);
        __syncthreads();
        if constexpr (FULL) {
            if (stages && t + sr < p.t1) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float y = fmaf(Dv[j], u_now.get(j), dx[sr * PAD + 8 * sv + j].x);
                    if (a.z) {
                        const float zv = z_now.get(j);
                        y *= zv * sigmoid_f(zv);
                    }
                    o[j] = y;
                }
                Raw8<T>::store(yp + (int64_t)(t + sr) * a.E, o);
            }
            u_now = u_next;
            z_now = z_next;
        }
    }

    if constexpr (FULL) {
        if (p.t1 == p.s1) {
            if constexpr (PACKED) {
                const int slot = slot_at(sl, sl.slot_of[p.s1 - 1]);
                if (slot >= 0 && live) store_h(a.final_state + slot * st_all + st);
            } else if (live && a.final_state) {
                store_h(a.final_state + p.r * st_all + st);
            }
        }
    } else if (MODE == kLocal && live) {
        store_h(ws.h + p.idx * st_all + st);
        if (q == 0) ws.sdt[p.idx * a.E + e] = sdt;
    }
}

constexpr int kWarpsWanted = 148 * 8;   // per device, below which rows are cut
constexpr int kPieceLeast = 128;        // rows; a shorter piece costs more to join than it gains

// Rows per piece, or no cut (the rows' count): one sequence that had all the
// rows would get as many pieces as fill the device; sequences shorter than a
// piece stay whole.
int piece_rows(int nseq, int rows, int E, int N, int G)
{
    const int ch = kThreads / diag_lanes(N);
    const int64_t ctas = (int64_t)((E / G + ch - 1) / ch) * G;
    const int64_t pieces = kWarpsWanted / (ctas * (kThreads / 32));
    if (pieces < 2) return rows;
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
    constexpr int smem = (int)sizeof(Smem<LPC>);
    static_assert(smem <= 48 * 1024, "no opt-in needed");
    const int per_group = a.E / a.G, CH = Tile<LPC>::CH;
    const dim3 grid((unsigned)pieces, (unsigned)((per_group + CH - 1) / CH * a.G));
    diag_scan_kernel<T, LPC, PACKED, MODE, CUT><<<grid, kThreads, smem, s>>>(a, seg, pieces);
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
cudaError_t launch_t(const DiagArgs& a, int seg, cudaStream_t s)
{
    switch (diag_lanes(a.N)) {
        case 1: return launch_lpc<T, 1, PACKED, MODE>(a, seg, s);
        case 2: return launch_lpc<T, 2, PACKED, MODE>(a, seg, s);
        case 4: return launch_lpc<T, 4, PACKED, MODE>(a, seg, s);
        case 8: return launch_lpc<T, 8, PACKED, MODE>(a, seg, s);
        default: return launch_lpc<T, 16, PACKED, MODE>(a, seg, s);
    }
}

}  // namespace

size_t diag_scan_workspace_bytes(int nseq, int rows, int E, int N, int G)
{
    const int seg = piece_rows(nseq, rows, E, N, G);
    if (seg >= rows) return 0;
    // packed or dense: a dense batch has at most one short piece per sequence
    return cut_ws_bytes(nseq, nseq + ((int64_t)rows - 1) / seg + 1, E, N);
}

cudaError_t launch_diag_scan(const DiagArgs& a, cudaStream_t s)
{
    const int seg = piece_rows(a.nseq, a.rows, a.E, a.N, a.G);
    if (a.sl.cu) return a.bf16 ? launch_t<__nv_bfloat16, true, kOutput>(a, seg, s) : launch_t<float, true, kOutput>(a, seg, s);
    return a.bf16 ? launch_t<__nv_bfloat16, false, kOutput>(a, seg, s) : launch_t<float, false, kOutput>(a, seg, s);
}

cudaError_t launch_diag_ckpt(const DiagArgs& a, int seg, cudaStream_t s)
{
    return a.bf16 ? launch_t<__nv_bfloat16, false, kCkpt>(a, seg, s) : launch_t<float, false, kCkpt>(a, seg, s);
}

size_t diag_cut_bytes(int nseq, int64_t pieces, int E, int N) { return cut_ws_bytes(nseq, pieces, E, N); }

}  // namespace ssd
