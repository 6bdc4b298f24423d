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
// before every 4th row (16 bytes per token and channel at N = 16; HBM has room
// for them, and keeping every 8th costs the walk of 4 rows in 8 once more);
// this one walks the rows from the end, 4 at a time: forward from the kept
// state, with a and a h of the 4 rows in registers (w_t = g_t (a_t h_{t-1}),
// so h itself is not needed after its products with C and p), then back.  Rows
// lie in pairs, as in the forward scan, for the packed instructions.
//
// Rows in pieces.  The kernel's time is that of its fullest SM, and a piece's
// walk needs G behind it.  The forward walk has the decays at hand, so it also
// leaves each piece's part of G at its start, sum_t (a_s .. a_t) C_t p_t, for
// two more products per element; folded over the pieces behind, that is the
// piece's G, and the rows can be cut as finely as balances the device.
//
// Sums go both ways, over states (gB, w A, and y for dz) and over channels
// (dB, dC), so a thread owns a patch of 2 channels x 4 states (diag_tile.cuh):
// both sums begin in registers.  Each is finished by an exchange that halves
// the values a lane keeps with every step, and where it can without a
// selection: a lane's slots hold its states in an order of its own (slot k is
// state k ^ m, m from the lane's channel number), so that what it keeps and
// what it sends are the same slots in every lane.  B and C lie in shared
// memory in all four orders.  The warps' channel sums meet in shared memory,
// the CTAs' in the workspace, where a last kernel adds them in a fixed order:
// no atomics, the same bits each run.  dA, dD and ddt_bias are summed the same
// way per piece.
//
// The walk is four fifths of the work here, so all four warps walk (half of
// them feeding the others, as in the forward scan, took 1700 us where this
// takes 990).  Between two tiles' walks one half of the CTA lays
// out the next tile (u, dt_raw, dy and z by cp.async a tile ahead; dt, x and p
// formed once per token and channel) while the other finishes du, ddt_raw and
// dz of the last one from its sums, in 16-byte vectors.
//
// 8 x 2048 tokens of 2560 gated bf16 channels, 16 states: 1440 us for the call,
// about 960 of them here, the forward walk 468, the sums 15.  Bound by instruction issue (27 per token, channel
// and state, 53% of the issue slots: 168 registers hold the 4 rows, so 12
// warps share an SM) and by shared memory's wavefronts (54%), not by HBM.
#include "diag_tile.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kHalf = kThreads / 2;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T, int LPC> struct Smem {
    using TL = DiagTile<LPC, kWarps>;
    static constexpr int PAIRS = TL::TT / 2;
    float4 tile[2][PAIRS][TL::CH];            // dt, dt', x, x' of two rows
    float2 p[2][PAIRS][TL::CH];
    float4 B[PAIRS][2][4][LPC], C[PAIRS][2][4][LPC];   // [half][order][lane]: b0, b0', b1, b1'; b2, ..
    T raw[2][4][TL::TT][TL::CH];              // u, dt_raw, dy, z
};

// Kept states and partial sums in the workspace.
struct BwdWs {
    float *ckpt, *cut, *gl, *gsdt, *dA, *dD, *dbias, *bc;
};

// A thread's 4 states in the order of its slots (and back: the order is its
// own inverse).
__device__ inline float4 order4(float4 v, int m)
{
    if (m & 2) v = make_float4(v.z, v.w, v.x, v.y);
    if (m & 1) v = make_float4(v.y, v.x, v.w, v.z);
    return v;
}

// keep + the partner's send, d lanes away
__device__ inline float ex(float keep, float send, int d) { return keep + __shfl_xor_sync(0xffffffffu, send, d); }
__device__ inline float2 ex(float2 keep, float2 send, int d) { return make_float2(ex(keep.x, send.x, d), ex(keep.y, send.y, d)); }

// Sums over a warp's channel lanes of a pair of rows' 4 slots: slots 0 and 2,
// then slot 0, are kept; of 8 lanes and more, a row; put(row, slot, sum).
template <int LPC, typename PUT>
__device__ inline void channel_sum(const float2 (&s)[4], int cg, PUT put)
{
    constexpr int NL = 32 / LPC;
    float2 v = ex(s[0], s[1], LPC);
    const float2 v2 = ex(s[2], s[3], LPC);
    if constexpr (NL == 2) {
        put(0, 0, v.x);
        put(1, 0, v.y);
        put(0, 2, v2.x);
        put(1, 2, v2.y);
    } else {
        v = ex(v, v2, 2 * LPC);
        if constexpr (NL == 4) {
            put(0, 0, v.x);
            put(1, 0, v.y);
        } else {
            const int up = cg >> 2 & 1;
            float one = ex(up ? v.y : v.x, up ? v.x : v.y, 4 * LPC);
#pragma unroll
            for (int o = 8; o < NL; o <<= 1) one = ex(one, one, o * LPC);
            put(up, 0, one);
        }
    }
}

template <typename T, int LPC>
__global__ void __launch_bounds__(kThreads, 3) diag_bwd_kernel(const DiagBwdArgs ba, const BwdWs ws, int seg)
{
    using TL = DiagTile<LPC, kWarps>;
    constexpr int NL = TL::NL, CH = TL::CH, NP = TL::NP, VPR = TL::VPR, TT = TL::TT, PAIRS = TT / 2;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem<T, LPC>& sm = *reinterpret_cast<Smem<T, LPC>*>(smem_raw);
    // the walk's results: objects of their own, so that its reads of other
    // rows need not wait for these writes
    __shared__ __align__(16) float gb_sum[TT][CH], wa_sum[TT][CH], y_sum[TT][CH];
    __shared__ float2 red[kWarps][TT][NP];      // dB, dC of each warp's channels
    __shared__ float2 tails[8][PAIRS * VPR];    // dD, ddt_bias of the piece, by pair of rows and vector
    const DiagArgs& a = ba.f;

    const int ntiles = channel_tiles(a.E, a.G, CH) * a.G;
    const int piece = (int)(blockIdx.x / ntiles), ytile = blockIdx.x - piece * ntiles;
    Piece p;
    find_piece_dense(piece, a.L, seg, p);
    const ChannelTile ct(a.E, a.G, CH, ytile);
    const int e0 = ct.e0, e_end = ct.e_end;
    const int64_t st_all = (int64_t)a.E * a.N;
    const int ntile = (p.t1 - p.t0 + TT - 1) / TT;
    const bool gated = a.z != nullptr;
    const int tid = threadIdx.x;
    const bool lower = tid < kHalf;
    // tile w of the walk, which goes from the end
    auto tile_row = [&](int w) { return p.t0 + (ntile - 1 - w) * TT; };

    // Each half of the CTA shares the tile out: item i is vector i % VPR of
    // the pair of rows i / VPR.
    constexpr int ITEMS = PAIRS * VPR, PER = (ITEMS + kHalf - 1) / kHalf;
    const int half_id = lower ? tid : tid - kHalf;
    auto fetch = [&](int w) {      // the lower half: tile w, on its way
        auto& raw = sm.raw[w & 1];
        if (w < ntile)
#pragma unroll
            for (int k = 0; k < 2 * PER; ++k) {
                const int i = half_id + (k >> 1) * kHalf, r = 2 * (i / VPR) + (k & 1), c = 8 * (i % VPR);
                const int64_t row = tile_row(w) + r;
                if (i < ITEMS && row < p.t1 && e0 + c < e_end) {
                    cp_row8(&raw[0][r][c], static_cast<const T*>(a.u) + row * a.us + e0 + c);
                    cp_row8(&raw[1][r][c], static_cast<const T*>(a.dt) + row * a.dts + e0 + c);
                    cp_row8(&raw[2][r][c], static_cast<const T*>(ba.dy) + row * a.E + e0 + c);
                    if (gated) cp_row8(&raw[3][r][c], static_cast<const T*>(a.z) + row * a.zs + e0 + c);
                }
            }
        cp_commit();
    };
    auto lay_out = [&](int w) {    // the lower half
        cp_wait_all();             // a thread reads back what it copied itself
        auto& raw = sm.raw[w & 1];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = half_id + k * kHalf, pr = i / VPR, c = 8 * (i % VPR);
            if (i >= ITEMS) break;
            const bool in = e0 + c < e_end;   // rows and channels outside change nothing
            const bool ok0 = in && tile_row(w) + 2 * pr < p.t1, ok1 = in && tile_row(w) + 2 * pr + 1 < p.t1;
            const Raw8<T> u0 = smem_row8(&raw[0][2 * pr][c]), u1 = smem_row8(&raw[0][2 * pr + 1][c]);
            const Raw8<T> v0 = smem_row8(&raw[1][2 * pr][c]), v1 = smem_row8(&raw[1][2 * pr + 1][c]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float bias = in && a.dt_bias ? __ldg(a.dt_bias + e0 + c + j) : 0.0f;
                const float2 dt = softplus_pair(make_float2(v0.get(j) + bias, v1.get(j) + bias));
                sm.tile[w & 1][pr][TL::col16(c + j, pr)] =
                    make_float4(ok0 ? dt.x : 0.0f, ok1 ? dt.y : 0.0f, ok0 ? dt.x * u0.get(j) : 0.0f, ok1 ? dt.y * u1.get(j) : 0.0f);
            }
            const Raw8<T> g0 = smem_row8(&raw[2][2 * pr][c]), g1 = smem_row8(&raw[2][2 * pr + 1][c]);
            const Raw8<T> z0 = smem_row8(&raw[3][2 * pr][c]), z1 = smem_row8(&raw[3][2 * pr + 1][c]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float2 g = make_float2(g0.get(j), g1.get(j));
                if (gated) {
                    g.x *= z0.get(j) * sigmoid_f(z0.get(j));
                    g.y *= z1.get(j) * sigmoid_f(z1.get(j));
                }
                sm.p[w & 1][pr][TL::col8(c + j, pr)] = make_float2(ok0 ? g.x : 0.0f, ok1 ? g.y : 0.0f);
            }
        }
    };
    // B and C: quads of states of pairs of rows, to the upper half
    constexpr int QUADS = (PAIRS * LPC + kHalf - 1) / kHalf;
    float bv[QUADS][2][4], cv[QUADS][2][4];
    auto fetch_bc = [&](int w) {
        const T* Bp = static_cast<const T*>(a.B) + (int64_t)ct.group * a.N;
        const T* Cp = static_cast<const T*>(a.C) + (int64_t)ct.group * a.N;
#pragma unroll
        for (int k = 0; k < QUADS; ++k) {
            const int at = half_id + k * kHalf, n = 4 * (at % LPC);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t row = tile_row(w) + 2 * (at / LPC) + h;
#pragma unroll
                for (int i = 0; i < 4; ++i) bv[k][h][i] = cv[k][h][i] = 0.0f;
                if (w < ntile && at < PAIRS * LPC && row < p.t1 && n < a.N) {
                    load4(Bp + row * a.bcs + n, a.bc_aligned, bv[k][h]);
                    load4(Cp + row * a.bcs + n, a.bc_aligned, cv[k][h]);
                }
            }
        }
    };
    auto lay_out_bc = [&] {
#pragma unroll
        for (int k = 0; k < QUADS; ++k) {
            const int at = half_id + k * kHalf, pr = at / LPC, q = at % LPC;
            if (at < PAIRS * LPC)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    sm.B[pr][0][m][q] = make_float4(bv[k][0][m], bv[k][1][m], bv[k][0][1 ^ m], bv[k][1][1 ^ m]);
                    sm.B[pr][1][m][q] = make_float4(bv[k][0][2 ^ m], bv[k][1][2 ^ m], bv[k][0][3 ^ m], bv[k][1][3 ^ m]);
                    sm.C[pr][0][m][q] = make_float4(cv[k][0][m], cv[k][1][m], cv[k][0][1 ^ m], cv[k][1][1 ^ m]);
                    sm.C[pr][1][m][q] = make_float4(cv[k][0][2 ^ m], cv[k][1][2 ^ m], cv[k][0][3 ^ m], cv[k][1][3 ^ m]);
                }
        }
    };
    auto finish = [&](int w) {     // the upper half
        const int t = tile_row(w);
        auto& raw = sm.raw[w & 1];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = half_id + k * kHalf, pr = i / VPR, c = 8 * (i % VPR);
            if (i >= ITEMS || t + 2 * pr >= p.t1 || e0 + c >= e_end) break;
            float dt[2][8], pv[2][8], sD[8], sb[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 d = *reinterpret_cast<const float2*>(&sm.tile[w & 1][pr][TL::col16(c + j, pr)]);
                const float2 g = sm.p[w & 1][pr][TL::col8(c + j, pr)];
                dt[0][j] = d.x; dt[1][j] = d.y;
                pv[0][j] = g.x; pv[1][j] = g.y;
                sD[j] = sb[j] = 0.0f;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = 2 * pr + h;
                if (t + r >= p.t1) break;
                const int64_t o = (int64_t)(t + r) * a.E + e0 + c;
                const Raw8<T> u = smem_row8(&raw[0][r][c]), v = smem_row8(&raw[1][r][c]);
                float gb[8], wa[8], out[8], Dv[8];
                *reinterpret_cast<float4*>(gb) = *reinterpret_cast<const float4*>(&gb_sum[r][c]);
                *reinterpret_cast<float4*>(gb + 4) = *reinterpret_cast<const float4*>(&gb_sum[r][c + 4]);
                *reinterpret_cast<float4*>(wa) = *reinterpret_cast<const float4*>(&wa_sum[r][c]);
                *reinterpret_cast<float4*>(wa + 4) = *reinterpret_cast<const float4*>(&wa_sum[r][c + 4]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    Dv[j] = a.D ? __ldg(a.D + e0 + c + j) : 0.0f;
                    const float bias = a.dt_bias ? __ldg(a.dt_bias + e0 + c + j) : 0.0f;
                    const float uv = u.get(j);
                    out[j] = fmaf(Dv[j], pv[h][j], dt[h][j] * gb[j]);
                    wa[j] = fmaf(uv, gb[j], wa[j] * kLn2) * sigmoid_f(v.get(j) + bias);
                    sD[j] = fmaf(uv, pv[h][j], sD[j]);
                    sb[j] += wa[j];
                }
                Raw8<T>::store(static_cast<T*>(ba.du) + o, out);
                Raw8<T>::store(static_cast<T*>(ba.ddt) + o, wa);
                if (gated) {
                    const Raw8<T> dy = smem_row8(&raw[2][r][c]), z = smem_row8(&raw[3][r][c]);
                    *reinterpret_cast<float4*>(gb) = *reinterpret_cast<const float4*>(&y_sum[r][c]);
                    *reinterpret_cast<float4*>(gb + 4) = *reinterpret_cast<const float4*>(&y_sum[r][c + 4]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float zv = z.get(j);
                        out[j] = dy.get(j) * fmaf(Dv[j], u.get(j), gb[j]) * dsilu_f(zv, sigmoid_f(zv));
                    }
                    Raw8<T>::store(static_cast<T*>(ba.dz) + o, out);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float2 s = tails[j][i];   // this thread's alone
                s.x += sD[j];
                s.y += sb[j];
                tails[j][i] = s;
            }
        }
    };
    auto sum_warps = [&](int w) {  // the lower half
        const int t = tile_row(w), rows = min(TT, p.t1 - t);
        for (int k = half_id; k < rows * NP; k += kHalf) {
            const int row = k / NP, n = k % NP;
            if (n < a.N) {
                float2 s = red[0][row][n];
#pragma unroll
                for (int i = 1; i < kWarps; ++i) {
                    s.x += red[i][row][n].x;
                    s.y += red[i][row][n].y;
                }
                reinterpret_cast<float2*>(ws.bc)[((int64_t)ytile * a.rows + t + row) * a.N + n] = s;
            }
        }
    };
    for (int i = tid; i < 8 * ITEMS; i += kThreads) tails[i / ITEMS][i % ITEMS] = make_float2(0.0f, 0.0f);
    if (lower) fetch(0);
    else fetch_bc(0);

    const int lane = tid & 31, warp = tid >> 5;
    const int q = lane % LPC, cg = lane / LPC, n0 = 4 * q;
    const int m = cg & (NL >= 4 ? 3 : 1);          // the order of this lane's slots
    int cl[2];
    int64_t st[2];
    bool live[2];
    float A2[2][4], G[2][4];
    float2 dA[2][4];                               // of the pairs' first and second rows
    auto put4 = [&](float4 v, float (&o)[4]) {
        v = order4(v, m);
        o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
    };
    const int64_t last = p.first + pieces_per(a.L, seg) - 1;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        cl[j] = TL::channel(warp, lane, j);
        live[j] = e0 + cl[j] < e_end && n0 < a.N;
        st[j] = (int64_t)(e0 + cl[j]) * a.N + n0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            A2[j][k] = G[j][k] = 0.0f;
            dA[j][k] = make_float2(0.0f, 0.0f);
        }
        if (!live[j]) continue;
        put4(decay_rate(__ldg(reinterpret_cast<const float4*>(a.A + st[j]))), A2[j]);
        // G behind the piece's last row: dfinal, folded over the pieces behind
        if (ba.dfinal) put4(*reinterpret_cast<const float4*>(ba.dfinal + p.r * st_all + st[j]), G[j]);
        for (int64_t i = last; i > p.idx; --i) {
            const float sdt = ws.gsdt[i * a.E + e0 + cl[j]];
            float g[4];
            put4(*reinterpret_cast<const float4*>(ws.gl + i * st_all + st[j]), g);
#pragma unroll
            for (int k = 0; k < 4; ++k) G[j][k] = fmaf(ex2(A2[j][k] * sdt), G[j][k], g[k]);
        }
    }
    // the state before group g of 4 rows, counted from the piece's start
    const int64_t ck0 = (int64_t)p.r * ckpts_of(a.L) + (p.t0 - p.s0) / kDiagCkpt;
    float4 kept[2];
    auto fetch_kept = [&](int g) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            kept[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (live[j]) kept[j] = __ldcs(reinterpret_cast<const float4*>(ws.ckpt + (ck0 + g) * st_all + st[j]));
        }
    };
    static_assert(kDiagCkpt == 4, "the walk takes a group of 4 rows from a kept state");
    fetch_kept((p.t1 - p.t0 - 1) / 4);
    for (int w = 0; w < ntile; ++w) {
        const int buf = w & 1, t = tile_row(w);
        if (lower) {
            lay_out(w);
            if (w > 0) sum_warps(w - 1);
        } else {
            lay_out_bc();
            if (w > 0) finish(w - 1);
        }
        __syncthreads();
        if (lower) fetch(w + 1);
        else fetch_bc(w + 1);
#pragma unroll 1
        for (int gr = (min(TT, p.t1 - t) - 1) / 4; gr >= 0; --gr) {
            float h[2][4];
            put4(kept[0], h[0]);
            put4(kept[1], h[1]);
            const int before = (t - p.t0) / 4 + gr - 1;
            if (before >= 0) fetch_kept(before);
            // forward over the 4 rows
            float2 av[2][2][4], qv[2][2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int pr = 2 * gr + i;
                const float4 bb[2] = {sm.B[pr][0][m][q], sm.B[pr][1][m][q]}, cc[2] = {sm.C[pr][0][m][q], sm.C[pr][1][m][q]};
                float2 sC[4], ys[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 d = sm.tile[buf][pr][TL::col16(cl[j], pr)];
                    const float2 pp = sm.p[buf][pr][TL::col8(cl[j], pr)];
                    const float2 dd = make_float2(d.x, d.y), xx = make_float2(d.z, d.w);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 b2 = k & 1 ? make_float2(bb[k >> 1].z, bb[k >> 1].w) : make_float2(bb[k >> 1].x, bb[k >> 1].y);
                        const float2 c2 = k & 1 ? make_float2(cc[k >> 1].z, cc[k >> 1].w) : make_float2(cc[k >> 1].x, cc[k >> 1].y);
                        av[i][j][k] = make_float2(ex2(A2[j][k] * dd.x), ex2(A2[j][k] * dd.y));
                        const float2 xb = pk_mul(xx, b2);
                        const float q0 = av[i][j][k].x * h[j][k], h0 = q0 + xb.x;
                        const float q1 = av[i][j][k].y * h0, h1 = q1 + xb.y;
                        qv[i][j][k] = make_float2(q0, q1);
                        h[j][k] = h1;
                        const float2 hh = make_float2(h0, h1);
                        sC[k] = j ? pk_fma(hh, pp, sC[k]) : pk_mul(hh, pp);
                        if (gated) ys[j] = k ? pk_fma(hh, c2, ys[j]) : pk_mul(hh, c2);
                    }
                }
                channel_sum<LPC>(sC, cg, [&](int row, int slot, float v) { red[warp][2 * pr + row][n0 + (slot ^ m)].y = v; });
                if (gated) {
                    // over a channel's lanes: slot 0's channel is kept (diag_tile.cuh), then a row
                    const float2 y = ex(ys[0], ys[1], LPC / 2);
                    if constexpr (LPC >= 4) {
                        const int odd = q & 1;
                        float v = ex(odd ? y.y : y.x, odd ? y.x : y.y, 1);
#pragma unroll
                        for (int o = 2; o < LPC / 2; o <<= 1) v = ex(v, v, o);
                        y_sum[2 * pr + odd][cl[0]] = v;
                    } else {
                        y_sum[2 * pr][cl[0]] = y.x;
                        y_sum[2 * pr + 1][cl[0]] = y.y;
                    }
                }
            }
            // and back
#pragma unroll
            for (int i = 1; i >= 0; --i) {
                const int pr = 2 * gr + i;
                const float4 bb[2] = {sm.B[pr][0][m][q], sm.B[pr][1][m][q]}, cc[2] = {sm.C[pr][0][m][q], sm.C[pr][1][m][q]};
                float2 sB[4], gb[2], wa[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 d = sm.tile[buf][pr][TL::col16(cl[j], pr)];
                    const float2 pp = sm.p[buf][pr][TL::col8(cl[j], pr)];
                    const float2 dd = make_float2(d.x, d.y), xx = make_float2(d.z, d.w);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 b2 = k & 1 ? make_float2(bb[k >> 1].z, bb[k >> 1].w) : make_float2(bb[k >> 1].x, bb[k >> 1].y);
                        const float2 c2 = k & 1 ? make_float2(cc[k >> 1].z, cc[k >> 1].w) : make_float2(cc[k >> 1].x, cc[k >> 1].y);
                        const float g1 = fmaf(c2.y, pp.y, G[j][k]);
                        const float g0 = fmaf(c2.x, pp.x, av[i][j][k].y * g1);
                        G[j][k] = av[i][j][k].x * g0;
                        const float2 gg = make_float2(g0, g1);
                        gb[j] = k ? pk_fma(gg, b2, gb[j]) : pk_mul(gg, b2);
                        sB[k] = j ? pk_fma(gg, xx, sB[k]) : pk_mul(gg, xx);
                        const float2 w2 = pk_mul(gg, qv[i][j][k]);
                        dA[j][k] = pk_fma(w2, dd, dA[j][k]);
                        // (scalar: a pair of A would have to be copied together)
                        wa[j] = k ? make_float2(fmaf(w2.x, A2[j][k], wa[j].x), fmaf(w2.y, A2[j][k], wa[j].y))
                                  : make_float2(w2.x * A2[j][k], w2.y * A2[j][k]);
                    }
                }
                channel_sum<LPC>(sB, cg, [&](int row, int slot, float v) { red[warp][2 * pr + row][n0 + (slot ^ m)].x = v; });
                const float2 vg = ex(gb[0], gb[1], LPC / 2), vw = ex(wa[0], wa[1], LPC / 2);
                if constexpr (LPC >= 4) {
                    const bool odd = q & 1;
                    float2 v = ex(odd ? vw : vg, odd ? vg : vw, 1);
#pragma unroll
                    for (int o = 2; o < LPC / 2; o <<= 1) v = ex(v, v, o);
                    float(*to)[CH] = odd ? wa_sum : gb_sum;
                    to[2 * pr][cl[0]] = v.x;
                    to[2 * pr + 1][cl[0]] = v.y;
                } else {
                    gb_sum[2 * pr][cl[0]] = vg.x;
                    gb_sum[2 * pr + 1][cl[0]] = vg.y;
                    wa_sum[2 * pr][cl[0]] = vw.x;
                    wa_sum[2 * pr + 1][cl[0]] = vw.y;
                }
            }
        }
        __syncthreads();
    }
    if (lower) sum_warps(ntile - 1);
    else finish(ntile - 1);
    __syncthreads();
    for (int c = tid; c < e_end - e0; c += kThreads) {
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int r = 0; r < PAIRS; ++r) {
            const float2 v = tails[c & 7][r * VPR + (c >> 3)];
            s.x += v.x;
            s.y += v.y;
        }
        ws.dD[p.idx * a.E + e0 + c] = s.x;
        ws.dbias[p.idx * a.E + e0 + c] = s.y;
    }

#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (!live[j]) continue;
        if (p.t0 == p.s0 && ba.dinit)
            *reinterpret_cast<float4*>(ba.dinit + p.r * st_all + st[j]) = order4(make_float4(G[j][0], G[j][1], G[j][2], G[j][3]), m);
        *reinterpret_cast<float4*>(ws.dA + p.idx * st_all + st[j]) =
            order4(make_float4(dA[j][0].x + dA[j][0].y, dA[j][1].x + dA[j][1].y, dA[j][2].x + dA[j][2].y, dA[j][3].x + dA[j][3].y), m);
    }
}

// The partial sums, in a fixed order, one launch for all.  The first bc_blocks
// CTAs: dB and dC, over a group's channel tiles of bc [G][tiles][rows][N].  The
// others: 32 columns each of dA, then dD, then ddt_bias [pieces][cols], 8 lanes
// of pieces joined in shared memory.
struct SumArgs {
    const float2* bc;
    const float* part[3];
    float* out[3];
    int64_t cols[3];
    void *dB, *dC;
    int64_t rows, pieces, bc_blocks;
    int tiles, N, G;
};
constexpr int kSumThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kSumThreads) diag_sum_kernel(const SumArgs a)
{
    __shared__ float sums[8][32];
    if (blockIdx.x < a.bc_blocks) {
        const int64_t per = a.rows * a.N;
        const int64_t at = (int64_t)blockIdx.x * kSumThreads + threadIdx.x;
        if (at >= per * a.G) return;
        const int64_t g = at / per, i = at - g * per;
        const float2* src = a.bc + g * a.tiles * per + i;
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll 8
        for (int k = 0; k < a.tiles; ++k) {
            const float2 v = __ldcs(src + k * per);
            s.x += v.x;
            s.y += v.y;
        }
        const int64_t row = i / a.N, o = (row * a.G + g) * a.N + (i - row * a.N);
        static_cast<T*>(a.dB)[o] = io<T>::from_f(s.x);
        static_cast<T*>(a.dC)[o] = io<T>::from_f(s.y);
        return;
    }
    int64_t block = blockIdx.x - a.bc_blocks;
    int which = 0;
    while (block >= (a.cols[which] + 31) / 32) block -= (a.cols[which++] + 31) / 32;
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    const int64_t cols = a.cols[which], col = block * 32 + x;
    float s = 0.0f;
    if (col < cols)
        for (int64_t i = y; i < a.pieces; i += 8) s += a.part[which][i * cols + col];
    sums[y][x] = s;
    __syncthreads();
    if (y == 0 && col < cols) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sums[i][x];
        a.out[which][col] = s;
    }
}

// Rows per piece.  The forward walk pays for the pieces (306 us without, 468
// with them, at 8 x 2048 rows of 2560 channels), this kernel gains from them
// (1390 us whole, 2 or 3 CTAs on an SM for all of its time), so rows are cut
// where whole sequences make less than kLeastPerSm CTAs an SM.  An SM holds
// kPerSm at a time; the pieces are the longest of 512, 256, 128 and 64 rows that
// take the device up 2.5 times or more, else 64, and where those take it up less
// than 1.25 times, such as fit it at once (a few CTAs of a second round would
// take as long as the first).  The whole call, 8 x 2048 x 2560: 512 rows (2.9
// times) 1441 us, 192 1452, 320 1473, 96 1517, 64 1576; 4 x 2048 x 2560: 256
// rows 940, 160 962, 512 (1.4 times) 1000, and 384 (1.9 times), which the rule
// does not try, 898; 8 x 256 x 2048: 64 rows (2.3 times) 185, 96 210; 1 x
// 2048 x 1024: 64 rows (1.15 times) 141, 96 120, 192 162; 2 x 517 x 784: 64
// rows (0.95 times) 89, 96 112.
// No piece is longer than 512 rows, and each folds G over all behind it: from
// some 100000 rows a sequence on, that reading (E N 4 bytes a piece) grows with
// the square of the rows: 8.6 GB at 1 x 262144 x 1024, N = 16, twice what the
// kept states are.
constexpr int kLeastPerSm = 12;
constexpr int kPerSm = 3;
constexpr int kPieceMost = 512, kPieceLeast = 64;

int bwd_piece_rows(int b, int L, int E, int N, int G)
{
    const int64_t ctas = (int64_t)b * channel_tiles(E, G, kWarps * 64 / tile_lanes(N)) * G;
    const int64_t at_once = (int64_t)sm_count() * kPerSm;
    if (ctas >= (int64_t)sm_count() * kLeastPerSm) return L;
    int64_t seg = kPieceMost;
    while (seg > kPieceLeast && (seg >= L || 2 * ctas * L < 5 * at_once * seg)) seg /= 2;
    if (4 * ctas * L < 5 * at_once * seg) seg = (ctas * L + at_once * 32 - 1) / (at_once * 32) * 32;
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
    if (smem > 16 * 1024) {   // with the kernel's own arrays, beyond what needs no leave
        const cudaError_t e = cudaFuncSetAttribute((const void*)diag_bwd_kernel<T, LPC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    const int64_t grid = p.pieces * p.tiles * a.f.G;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    diag_bwd_kernel<T, LPC><<<(unsigned)grid, kThreads, smem, s>>>(a, ws, p.seg);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const DiagBwdArgs& args, const Plan& p, const BwdWs& ws, cudaStream_t s)
{
    DiagBwdArgs a = args;
    a.f.bc_aligned = bc_aligned(a.f, sizeof(T));
    cudaError_t e;
    switch (tile_lanes(a.f.N)) {
        case 2: e = launch_lpc<T, 2>(a, p, ws, s); break;
        case 4: e = launch_lpc<T, 4>(a, p, ws, s); break;
        case 8: e = launch_lpc<T, 8>(a, p, ws, s); break;
        default: e = launch_lpc<T, 16>(a, p, ws, s); break;
    }
    if (e != cudaSuccess) return e;
    const int64_t E = a.f.E, items = (int64_t)a.f.rows * a.f.N * a.f.G;
    SumArgs sum{reinterpret_cast<const float2*>(ws.bc), {ws.dA, ws.dD, ws.dbias}, {a.dA, a.dD, a.ddt_bias}, {E * a.f.N, E, E}, a.dB, a.dC,
                a.f.rows, p.pieces, (items + kSumThreads - 1) / kSumThreads, p.tiles, a.f.N, a.f.G};
    int64_t grid = sum.bc_blocks;
    for (const int64_t c : sum.cols) grid += (c + 31) / 32;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    diag_sum_kernel<T><<<(unsigned)grid, kSumThreads, 0, s>>>(sum);
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
    return e;
}

}  // namespace ssd
