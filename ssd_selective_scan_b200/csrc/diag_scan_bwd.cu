// diag_scan_bwd.cu -- gradients of the diagonal selective scan.
//
// With a_t = exp(dt_t A), x_t = dt_t u_t, p_t = dy_t SiLU(z_t) and g_t the
// gradient with respect to h_t, per channel e and state n:
//   g_t = C_t p_t + G_{t+1},   G_t = a_t g_t,   G_L = dfinal,   dinit = G_0,
//   dC_t[n] = sum_e h_t p_t,        dB_t[n] = sum_e g_t x_t,
//   gB_t = sum_n g_t B_t,           w_t = G_t h_{t-1},
//   du_t = D p_t + dt_t gB_t,       ddt_t = u_t gB_t + sum_n w_t A,
//   ddt_raw = ddt sigmoid(dt_raw + bias),   dA = sum_t w_t dt_t,
//   dD = sum_t u_t p_t,   dz_t = dy_t (sum_n h_t C_t + D u_t) SiLU'(z_t).
// The products need h and g of the same row, one recurrence running forward
// and one backward.  So a first kernel walks forward and leaves the state
// before every 8th row (8 bytes per token and channel at N = 16); this one
// walks the rows from the end, 8 at a time: forward from the kept state with
// the 8 decays and states in registers, then back over them.
//
// Sums go both ways, over states (gB, w A, and y for dz) and over channels
// (dB, dC), so a thread owns a patch of 2 channels x 4 states: both sums
// begin in registers, where a patch of one channel would send twice the
// values through the channel sum.  LPC lanes hold a channel's states, the
// other lanes of the warp other channels, and each sum is finished by an
// exchange that halves the values a lane keeps with every step (7 shuffles
// for 8 channel sums over 8 lanes, 3 for 4 state sums over 4).  The 4 warps'
// channel sums meet in shared memory, the CTAs' in the workspace, where a
// last kernel adds them in a fixed order: no atomics, the same bits each run.
// dA, dD and ddt_bias are summed the same way per piece.
//
// u, dt_raw, dy and z are copied to shared memory one tile ahead (cp.async);
// dt, x and p are formed from them once per token and channel, and the state
// sums return through the same places to the threads that write du, ddt_raw
// and dz in 16-byte vectors.
//
// Bound by instruction issue, not by HBM: per token, channel and state 2
// exponentials (one per walk) and about 20 other instructions.
#include "diag_tile.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T, int LPC> struct Smem {
    using TL = DiagTile<LPC, kWarps>;
    float4 tile[TL::TT][TL::CH];              // dt, x -> gB, p, w A
    float ysum[TL::TT][TL::CH];
    float4 B[TL::TT][LPC], C[TL::TT][LPC];
    float2 red[kWarps][TL::TT][TL::NP];       // dB, dC of each warp's channels
    T raw[2][4][TL::TT][TL::CH];              // u, dt_raw, dy, z
};

// Kept states and partial sums in the workspace.
struct BwdWs {
    float *ckpt, *cut, *gl, *gsdt, *dA, *dD, *dbias, *bc;
};

template <typename T, int LPC>
__global__ void __launch_bounds__(kThreads) diag_bwd_kernel(const DiagBwdArgs ba, const BwdWs ws, int seg)
{
    using TL = DiagTile<LPC, kWarps>;
    constexpr int NL = TL::NL, TT = TL::TT, VPR = TL::VPR, NP = TL::NP, NBC = TL::NBC;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem<T, LPC>& sm = *reinterpret_cast<Smem<T, LPC>*>(smem_raw);
    const DiagArgs& a = ba.f;

    Piece p;
    find_piece_dense(blockIdx.x, a.L, seg, p);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane % LPC, cg = lane / LPC;
    const ChannelTile ct(a.E, a.G, TL::CH, blockIdx.y);
    const int e0 = ct.e0, e_end = ct.e_end;
    const int n0 = 4 * q;
    const int64_t st_all = (int64_t)a.E * a.N;
    int cl[2], col[2];
    int64_t st[2];
    bool live[2];
    float2 A2[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        cl[j] = TL::channel(warp, lane, j);
        col[j] = TL::col16(cl[j], 0);
        live[j] = e0 + cl[j] < e_end && n0 < a.N;
        st[j] = (int64_t)(e0 + cl[j]) * a.N + n0;
        A2[j][0] = A2[j][1] = make_float2(0.0f, 0.0f);
        if (live[j]) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(a.A + st[j]));
            A2[j][0] = make_float2(v.x * kLog2e, v.y * kLog2e);
            A2[j][1] = make_float2(v.z * kLog2e, v.w * kLog2e);
        }
    }

    // G behind the piece's last row: dfinal, folded over the pieces behind
    float2 G[2][2], dA[2][2];
    const int64_t last = p.first + pieces_per(a.L, seg) - 1;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        G[j][0] = G[j][1] = dA[j][0] = dA[j][1] = make_float2(0.0f, 0.0f);
        if (!live[j]) continue;
        if (ba.dfinal) {
            const float4 v = *reinterpret_cast<const float4*>(ba.dfinal + p.r * st_all + st[j]);
            G[j][0] = make_float2(v.x, v.y);
            G[j][1] = make_float2(v.z, v.w);
        }
        for (int64_t i = last; i > p.idx; --i) {
            const float sdt = ws.gsdt[i * a.E + e0 + cl[j]];
            const float4 v = *reinterpret_cast<const float4*>(ws.gl + i * st_all + st[j]);
            G[j][0].x = fmaf(ex2(A2[j][0].x * sdt), G[j][0].x, v.x);
            G[j][0].y = fmaf(ex2(A2[j][0].y * sdt), G[j][0].y, v.y);
            G[j][1].x = fmaf(ex2(A2[j][1].x * sdt), G[j][1].x, v.z);
            G[j][1].y = fmaf(ex2(A2[j][1].y * sdt), G[j][1].y, v.w);
        }
    }

    // loading: vector sv of row sr of each tile
    const int sr = tid / VPR, sv = tid % VPR;
    const int ev = e0 + 8 * sv;
    const bool loads = tid < TL::NVEC && ev < e_end;
    float Dv[8], bias[8], dDs[8], dbs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        Dv[j] = loads && a.D ? a.D[ev + j] : 0.0f;
        bias[j] = loads && a.dt_bias ? a.dt_bias[ev + j] : 0.0f;
        dDs[j] = dbs[j] = 0.0f;
    }
    const T* Bp = static_cast<const T*>(a.B) + (int64_t)ct.group * a.N;
    const T* Cp = static_cast<const T*>(a.C) + (int64_t)ct.group * a.N;
    const bool gated = a.z != nullptr;

    auto fetch = [&](int t, int buf) {
        const int64_t row = t + sr;
        if (loads && row < p.t1) {
            cp_row8(&sm.raw[buf][0][sr][8 * sv], static_cast<const T*>(a.u) + row * a.us + ev);
            cp_row8(&sm.raw[buf][1][sr][8 * sv], static_cast<const T*>(a.dt) + row * a.dts + ev);
            cp_row8(&sm.raw[buf][2][sr][8 * sv], static_cast<const T*>(ba.dy) + row * a.E + ev);
            if (gated) cp_row8(&sm.raw[buf][3][sr][8 * sv], static_cast<const T*>(a.z) + row * a.zs + ev);
        }
        cp_commit();
    };
    float bq[NBC], cq[NBC];
    auto fetch_bc = [&](int t) {
#pragma unroll
        for (int i = 0; i < NBC; ++i) {
            const int k = tid + i * kThreads, row = k / NP, n = k % NP;
            const bool ok = k < TT * NP && t + row < p.t1 && n < a.N;
            bq[i] = ok ? ld_f(Bp + (int64_t)(t + row) * a.bcs + n) : 0.0f;
            cq[i] = ok ? ld_f(Cp + (int64_t)(t + row) * a.bcs + n) : 0.0f;
        }
    };
    auto raw8 = [&](int buf, int i) { return smem_row8(&sm.raw[buf][i][sr][8 * sv]); };

    const int ntile = (p.t1 - p.t0 + TT - 1) / TT;
    const int64_t ck0 = (int64_t)p.r * ckpts_of(a.L) + (p.t0 - p.s0) / kDiagCkpt;   // the piece's first kept state
    fetch(p.t0 + (ntile - 1) * TT, 0);
    fetch_bc(p.t0 + (ntile - 1) * TT);
    int buf = 0;
    for (int it = ntile - 1; it >= 0; --it, buf ^= 1) {
        const int t = p.t0 + it * TT;
        cp_wait_all();   // a thread reads back what it copied itself
        if (tid < TL::NVEC) {
            const bool ok = loads && t + sr < p.t1;
            const Raw8<T> u = raw8(buf, 0), v = raw8(buf, 1), dy = raw8(buf, 2), z = raw8(buf, 3);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (ok) {
                    f.x = softplus_series(v.get(j) + bias[j]);
                    f.y = f.x * u.get(j);
                    f.z = dy.get(j);
                    if (gated) f.z *= z.get(j) * sigmoid_f(z.get(j));
                }
                sm.tile[sr][TL::col16(8 * sv + j, 0)] = f;
            }
        }
#pragma unroll
        for (int i = 0; i < NBC; ++i) {
            const int k = tid + i * kThreads;
            if (k < TT * NP) {
                reinterpret_cast<float*>(sm.B)[k] = bq[i];
                reinterpret_cast<float*>(sm.C)[k] = cq[i];
            }
        }
        __syncthreads();
        if (it > 0) {
            fetch(t - TT, buf ^ 1);
            fetch_bc(t - TT);
        }

#pragma unroll 1
        for (int half = TT / kDiagCkpt - 1; half >= 0; --half) {
            const int r0 = half * kDiagCkpt;
            if (t + r0 >= p.t1) continue;
            // forward over 8 rows: decays and states
            float2 av[kDiagCkpt][2][2], hv[kDiagCkpt + 1][2][2];
            const float* ck = ws.ckpt + (ck0 + (it * TT + r0) / kDiagCkpt) * st_all;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (live[j]) v = __ldcs(reinterpret_cast<const float4*>(ck + st[j]));
                hv[0][j][0] = make_float2(v.x, v.y);
                hv[0][j][1] = make_float2(v.z, v.w);
            }
#pragma unroll
            for (int i = 0; i < kDiagCkpt; ++i) {
                const float4 b4 = sm.B[r0 + i][q];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 d = *reinterpret_cast<const float2*>(&sm.tile[r0 + i][col[j]]);
                    const float2 dd = make_float2(d.x, d.x), xx = make_float2(d.y, d.y);
                    const float2 s0 = pk_mul(A2[j][0], dd), s1 = pk_mul(A2[j][1], dd);
                    av[i][j][0] = make_float2(ex2(s0.x), ex2(s0.y));
                    av[i][j][1] = make_float2(ex2(s1.x), ex2(s1.y));
                    hv[i + 1][j][0] = pk_fma(av[i][j][0], hv[i][j][0], pk_mul(make_float2(b4.x, b4.y), xx));
                    hv[i + 1][j][1] = pk_fma(av[i][j][1], hv[i][j][1], pk_mul(make_float2(b4.z, b4.w), xx));
                }
            }
            // and back
#pragma unroll
            for (int i = kDiagCkpt - 1; i >= 0; --i) {
                const int row = r0 + i;
                const float4 b4 = sm.B[row][q], c4 = sm.C[row][q];
                const float2 b01 = make_float2(b4.x, b4.y), b23 = make_float2(b4.z, b4.w);
                const float2 c01 = make_float2(c4.x, c4.y), c23 = make_float2(c4.z, c4.w);
                float sn[4], sy[2];       // state sums: gB, w A of each channel; y
                float2 sB[2], sC[2];      // channel sums
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 d = sm.tile[row][col[j]];
                    const float2 pp = make_float2(d.z, d.z), xx = make_float2(d.y, d.y), dd = make_float2(d.x, d.x);
                    const float2 g0 = pk_fma(c01, pp, G[j][0]), g1 = pk_fma(c23, pp, G[j][1]);
                    const float2 gb = pk_fma(g0, b01, pk_mul(g1, b23));
                    sn[2 * j] = gb.x + gb.y;
                    if (j == 0) {
                        sB[0] = pk_mul(g0, xx); sB[1] = pk_mul(g1, xx);
                        sC[0] = pk_mul(hv[i + 1][j][0], pp); sC[1] = pk_mul(hv[i + 1][j][1], pp);
                    } else {
                        sB[0] = pk_fma(g0, xx, sB[0]); sB[1] = pk_fma(g1, xx, sB[1]);
                        sC[0] = pk_fma(hv[i + 1][j][0], pp, sC[0]); sC[1] = pk_fma(hv[i + 1][j][1], pp, sC[1]);
                    }
                    G[j][0] = pk_mul(av[i][j][0], g0);
                    G[j][1] = pk_mul(av[i][j][1], g1);
                    const float2 w0 = pk_mul(G[j][0], hv[i][j][0]), w1 = pk_mul(G[j][1], hv[i][j][1]);
                    dA[j][0] = pk_fma(w0, dd, dA[j][0]);
                    dA[j][1] = pk_fma(w1, dd, dA[j][1]);
                    const float2 wa = pk_fma(w0, A2[j][0], pk_mul(w1, A2[j][1]));
                    sn[2 * j + 1] = wa.x + wa.y;
                    if (gated) {
                        const float2 yy = pk_fma(hv[i + 1][j][0], c01, pk_mul(hv[i + 1][j][1], c23));
                        sy[j] = yy.x + yy.y;
                    }
                }
                float sc[8] = {sB[0].x, sB[0].y, sB[1].x, sB[1].y, sC[0].x, sC[0].y, sC[1].x, sC[1].y};
                int at = 0;
                scatter_sum<8, NL, LPC>(sc, cg, at);
#pragma unroll
                for (int k = 0; k < (NL < 8 ? 8 / NL : 1); ++k)
                    reinterpret_cast<float*>(&sm.red[warp][row][n0 + ((at + k) & 3)])[(at + k) >> 2] = sc[k];
                // every lane keeps the channel of its slot 0 (diag_tile.cuh)
                float v[2] = {sn[0] + __shfl_xor_sync(0xffffffffu, sn[2], LPC / 2), sn[1] + __shfl_xor_sync(0xffffffffu, sn[3], LPC / 2)};
                at = 0;
                scatter_sum<2, LPC / 2, 1>(v, q % (LPC / 2), at);
#pragma unroll
                for (int k = 0; k < (LPC == 2 ? 2 : 1); ++k) reinterpret_cast<float*>(&sm.tile[row][col[0]])[2 * (at + k) + 1] = v[k];
                if (gated) {
                    float y = sy[0] + __shfl_xor_sync(0xffffffffu, sy[1], LPC / 2);
#pragma unroll
                    for (int o = LPC / 4; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                    sm.ysum[row][col[0]] = y;
                }
            }
        }
        __syncthreads();
        // the loading threads finish their 8 channels of a row
        if (loads && t + sr < p.t1) {
            const Raw8<T> u = raw8(buf, 0), v = raw8(buf, 1), dy = raw8(buf, 2), z = raw8(buf, 3);
            float du[8], ddt[8], dz[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = TL::col16(8 * sv + j, 0);
                const float4 f = sm.tile[sr][c];
                const float uv = u.get(j);
                du[j] = fmaf(Dv[j], f.z, f.x * f.y);
                ddt[j] = fmaf(uv, f.y, f.w * kLn2) * sigmoid_f(v.get(j) + bias[j]);
                dDs[j] = fmaf(uv, f.z, dDs[j]);
                dbs[j] += ddt[j];
                if (gated) {
                    const float zv = z.get(j);
                    dz[j] = dy.get(j) * fmaf(Dv[j], uv, sm.ysum[sr][c]) * dsilu_f(zv, sigmoid_f(zv));
                }
            }
            const int64_t o = (int64_t)(t + sr) * a.E + ev;
            Raw8<T>::store(static_cast<T*>(ba.du) + o, du);
            Raw8<T>::store(static_cast<T*>(ba.ddt) + o, ddt);
            if (gated) Raw8<T>::store(static_cast<T*>(ba.dz) + o, dz);
        }
        const int rows = min(TT, p.t1 - t);
        for (int k = tid; k < rows * NP; k += kThreads) {
            const int row = k / NP, n = k % NP;
            if (n < a.N) {
                float2 s = sm.red[0][row][n];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    s.x += sm.red[w][row][n].x;
                    s.y += sm.red[w][row][n].y;
                }
                reinterpret_cast<float2*>(ws.bc)[((int64_t)blockIdx.y * a.rows + t + row) * a.N + n] = s;
            }
        }
    }

#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (!live[j]) continue;
        if (p.t0 == p.s0 && ba.dinit)
            *reinterpret_cast<float4*>(ba.dinit + p.r * st_all + st[j]) = make_float4(G[j][0].x, G[j][0].y, G[j][1].x, G[j][1].y);
        *reinterpret_cast<float4*>(ws.dA + p.idx * st_all + st[j]) = make_float4(dA[j][0].x, dA[j][0].y, dA[j][1].x, dA[j][1].y);
    }
    // dD, ddt_bias: over the tile's rows through shared memory
    __syncthreads();
    if (loads)
#pragma unroll
        for (int j = 0; j < 8; ++j) *reinterpret_cast<float2*>(&sm.tile[sr][8 * sv + j]) = make_float2(dDs[j], dbs[j]);
    __syncthreads();
    for (int c = tid; c < e_end - e0; c += kThreads) {
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int r = 0; r < TT; ++r) {
            const float2 v = *reinterpret_cast<const float2*>(&sm.tile[r][c]);
            s.x += v.x;
            s.y += v.y;
        }
        ws.dD[p.idx * a.E + e0 + c] = s.x;
        ws.dbias[p.idx * a.E + e0 + c] = s.y;
    }
}

// dB, dC: the sum over a group's channel tiles of part [G][tiles][rows][N].
template <typename T>
__global__ void __launch_bounds__(256) sum_bc_kernel(const float2* __restrict__ part, T* __restrict__ dB, T* __restrict__ dC, int tiles,
                                                     int64_t rows, int N, int G)
{
    const int64_t per = rows * N;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int g = blockIdx.y;
    if (i >= per) return;
    const float2* src = part + (int64_t)g * tiles * per + i;
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll 8
    for (int k = 0; k < tiles; ++k) {
        const float2 v = __ldcs(src + k * per);
        s.x += v.x;
        s.y += v.y;
    }
    const int64_t row = i / N, o = (row * G + g) * N + (i - row * N);
    dB[o] = io<T>::from_f(s.x);
    dC[o] = io<T>::from_f(s.y);
}

// Columns of part [parts][cols], 32 x 8 threads: 8 lanes of parts, joined in
// a fixed order.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ part, float* __restrict__ out, int64_t parts, int64_t cols)
{
    __shared__ float sums[8][32];
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (col < cols)
        for (int64_t i = threadIdx.y; i < parts; i += 8) s += part[i * cols + col];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && col < cols) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sums[i][threadIdx.x];
        out[col] = s;
    }
}

// Rows per piece.  The kernel's time is that of its fullest SM, so the rows
// are cut until the CTAs make kWaves of what the device holds at a time: a
// last, partly filled wave then costs little.
constexpr int kCtasAtATime = 148 * 2;
constexpr int kWaves = 6;
constexpr int kPieceLeast = 64;

int bwd_piece_rows(int b, int L, int E, int N, int G)
{
    const int64_t ctas = (int64_t)b * channel_tiles(E, G, kWarps * 64 / tile_lanes(N)) * G;
    const int64_t pieces = (kCtasAtATime * kWaves + ctas - 1) / ctas;
    if (pieces < 2) return L;
    int64_t seg = ((int64_t)L + pieces - 1) / pieces;
    seg = (seg + 31) / 32 * 32;
    if (seg < kPieceLeast) seg = kPieceLeast;
    return seg < L ? (int)seg : L;
}

struct Plan {
    int seg, tiles;
    int64_t pieces;
    size_t ckpt, cut, gl, gsdt, dA, dD, dbias, bc, total;   // byte offsets
};

Plan plan_of(int b, int L, int E, int N, int G)
{
    Plan p{};
    p.seg = bwd_piece_rows(b, L, E, N, G);
    p.pieces = (int64_t)b * pieces_per(L, p.seg);
    p.tiles = channel_tiles(E, G, kWarps * 64 / tile_lanes(N));
    const int walk = diag_ckpt_rows(b, L, E, N, G, p.seg);
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t state = (size_t)E * N * 4, parts = (size_t)p.pieces;
    p.ckpt = 0;
    p.cut = p.ckpt + up((size_t)b * ckpts_of(L) * state);
    p.gl = p.cut + (walk < L ? up(diag_cut_bytes(b, (int64_t)b * pieces_per(L, walk), E, N)) : 0);
    p.gsdt = p.gl + (p.seg < L ? up(parts * state) : 0);
    p.dA = p.gsdt + (p.seg < L ? up(parts * E * 4) : 0);
    p.dD = p.dA + up(parts * state);
    p.dbias = p.dD + up(parts * E * 4);
    p.bc = p.dbias + up(parts * E * 4);
    p.total = p.bc + up((size_t)p.tiles * G * b * L * N * 8);
    return p;
}

template <typename T, int LPC>
cudaError_t launch_lpc(const DiagBwdArgs& a, const Plan& p, const BwdWs& ws, cudaStream_t s)
{
    const int smem = (int)sizeof(Smem<T, LPC>);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute((const void*)diag_bwd_kernel<T, LPC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    diag_bwd_kernel<T, LPC><<<dim3((unsigned)p.pieces, (unsigned)(p.tiles * a.f.G)), kThreads, smem, s>>>(a, ws, p.seg);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const DiagBwdArgs& a, const Plan& p, const BwdWs& ws, cudaStream_t s)
{
    cudaError_t e;
    switch (tile_lanes(a.f.N)) {
        case 2: e = launch_lpc<T, 2>(a, p, ws, s); break;
        case 4: e = launch_lpc<T, 4>(a, p, ws, s); break;
        case 8: e = launch_lpc<T, 8>(a, p, ws, s); break;
        default: e = launch_lpc<T, 16>(a, p, ws, s); break;
    }
    if (e != cudaSuccess) return e;
    const int64_t per = (int64_t)a.f.rows * a.f.N;
    sum_bc_kernel<T><<<dim3((unsigned)((per + 255) / 256), (unsigned)a.f.G), 256, 0, s>>>(
        reinterpret_cast<const float2*>(ws.bc), static_cast<T*>(a.dB), static_cast<T*>(a.dC), p.tiles, a.f.rows, a.f.N, a.f.G);
    return cudaGetLastError();
}

}  // namespace

size_t diag_scan_bwd_workspace_bytes(int b, int L, int E, int N, int G) { return plan_of(b, L, E, N, G).total; }

cudaError_t launch_diag_scan_bwd(const DiagBwdArgs& a, cudaStream_t s)
{
    const Plan p = plan_of(a.f.nseq, a.f.L, a.f.E, a.f.N, a.f.G);
    uint8_t* base = static_cast<uint8_t*>(a.f.ws);
    auto at = [&](size_t off) { return reinterpret_cast<float*>(base + off); };
    const BwdWs ws{at(p.ckpt), at(p.cut), at(p.gl), at(p.gsdt), at(p.dA), at(p.dD), at(p.dbias), at(p.bc)};
    DiagArgs f = a.f;
    f.ws = ws.cut;
    f.dy = a.dy;
    f.ckpt = ws.ckpt;
    f.gl = ws.gl;
    f.gsdt = ws.gsdt;
    f.bseg = p.seg;
    cudaError_t e = launch_diag_ckpt(f, s);
    if (e == cudaSuccess) e = a.f.bf16 ? launch_t<__nv_bfloat16>(a, p, ws, s) : launch_t<float>(a, p, ws, s);
    auto sum = [&](const float* part, float* out, int64_t cols) {
        if (e != cudaSuccess) return;
        sum_parts_kernel<<<(unsigned)((cols + 31) / 32), dim3(32, 8), 0, s>>>(part, out, p.pieces, cols);
        e = cudaGetLastError();
    };
    sum(ws.dA, a.dA, (int64_t)a.f.E * a.f.N);
    sum(ws.dD, a.dD, a.f.E);
    sum(ws.dbias, a.ddt_bias, a.f.E);
    return e;
}

}  // namespace ssd
