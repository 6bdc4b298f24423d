// diag_tile.cuh -- how the diagonal scan's walks lay channels, states and rows
// over a CTA (forward, kept states, backward).
//
// A thread owns a patch of 2 channels x 4 states.  Shared memory serves a
// warp 32 words a cycle however few addresses differ, and a row's B and C
// are 8 words for each thread: a patch of two channels halves what they cost
// per state.  LPC lanes hold a channel's states (4 each), the NL = 32 / LPC
// groups of lanes different channels, so a warp covers 2 NL channels.
//
// A lane of the upper half of a channel's lanes holds its two channels in
// swapped order.  The first step of a sum over a channel's lanes then needs
// no selection: every lane keeps its slot 0 and sends its slot 1, which is
// the partner's slot 0.
#pragma once

#include "diag.cuh"
#include "diag.h"

namespace ssd {

template <int LPC, int WARPS> struct DiagTile {
    static constexpr int kThreads = 32 * WARPS;
    static constexpr int NL = 32 / LPC;                   // channel lanes of a warp
    static constexpr int CH = WARPS * 2 * NL;             // channels per CTA
    static constexpr int TT = LPC == 2 ? 8 : 16;          // rows per tile
    static constexpr int NP = 4 * LPC;                    // states, padded
    static constexpr int VPR = CH / 8;                    // 8-element vectors per row
    static constexpr int NVEC = TT * VPR;                 // ... per tile: at most one per thread
    static constexpr int NBC = (TT * NP + kThreads - 1) / kThreads;   // B (and C) elements per thread and tile
    static_assert(NVEC <= kThreads && TT % kDiagCkpt == 0, "");

    // the channel, within the CTA's, of slot j of a lane
    __device__ static int channel(int warp, int lane, int j)
    {
        const int q = lane % LPC, cg = lane / LPC;
        const int swap = LPC > 1 ? (q / (LPC / 2)) & 1 : 0;
        return warp * 2 * NL + 2 * cg + (j ^ swap);   // neighbours: 8 lanes read 4 adjacent entries
    }
    // Where channel c lies in a line of 16-byte (8-byte: col8) entries.  A
    // loading thread writes 8 adjacent channels; their order is turned by the
    // thread's number so that the threads of a wavefront write to different
    // banks.  `line` is the tile's row or pair of rows, VPR threads to each.
    __device__ static int col8(int c, int line)
    {
        const int turn = VPR == 8 ? (line & 1) << 2 : VPR == 4 ? (line & 3) << 1 : VPR == 2 ? line & 7 : (line >> 1) & 7;
        return (c & ~7) | (((c ^ (c >> 4)) & 7) ^ turn);
    }
    __device__ static int col16(int c, int line)
    {
        const int turn = VPR == 8 ? 0 : VPR == 4 ? (line & 1) << 2 : VPR == 2 ? (line & 3) << 1 : line & 7;
        return (c & ~7) | (((c ^ (c >> 3)) & 7) ^ turn);
    }
};

// lanes per channel: at least 2 (N <= 4 leaves the second lane's states empty:
// a tile of one-lane channels would be wider than a CTA's loads)
inline int tile_lanes(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

// The CTA's channels: tile y of the groups' tiles.
struct ChannelTile {
    int group, e0, e_end;
    __device__ ChannelTile(int E, int G, int CH, int y)
    {
        const int per = E / G, tiles = (per + CH - 1) / CH;
        group = y / tiles;
        e0 = group * per + (y - group * tiles) * CH;
        e_end = min(e0 + CH, (group + 1) * per);
    }
};
__host__ __device__ inline int channel_tiles(int E, int G, int CH) { return (E / G + CH - 1) / CH; }   // per group

__device__ inline void cp16(void* smem, const void* gmem)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem) : "memory");
}
__device__ inline void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ inline void cp_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// 8 adjacent elements to or from shared memory (16-byte aligned there).
template <typename T> __device__ inline void cp_row8(T* smem, const T* gmem)
{
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) cp16(smem + k * (16 / sizeof(T)), gmem + k * (16 / sizeof(T)));
}
template <typename T> __device__ inline Raw8<T> smem_row8(const T* p)
{
    Raw8<T> r;
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) r.q[k] = reinterpret_cast<const uint4*>(p)[k];
    return r;
}

}  // namespace ssd
