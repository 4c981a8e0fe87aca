// tiles.h -- the expert GEMMs' map from workgroups to (expert, token tile, feature tile).
#pragma once

#include "lanes.h"

namespace mxfp4 {

// Token tile `mtile` (tiles of TM rows, in expert order) -> expert, its first row and the
// tile's rows.
// False if the tile does not exist.  Experts are scanned 256 at a time, four consecutive ones
// per lane, so that up to 256 of them cost one round of loads (a round per 64 of them made a
// call of 2048 small tiles over 256 experts 1.35 times as long).
template <int TM>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ offs, int G, uint32_t mtile,
                                          int& g_out, int64_t& row0, int& rows)
{
    const int lane = threadIdx.x & 63;
    uint32_t run = 0;
    for (int g0 = 0; g0 < G; g0 += 256) {
        const int h = g0 + 4 * lane;
        int32_t r[5];
#pragma unroll
        for (int i = 0; i < 5; ++i)
            r[i] = offs[min(h + i, G)];
        uint32_t nt[4], own = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            own += nt[i] = (uint32_t)(r[i + 1] - r[i] + TM - 1) / TM;
        const uint32_t incl = wave_scan(own);
        // this lane's expert that has the tile, if one does
        uint32_t first = run + incl - own, at = 0;
        int g = -1;
        int32_t base = 0, m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (mtile >= first && mtile < first + nt[i]) {
                g = h + i;
                at = mtile - first;
                base = r[i];
                m = r[i + 1] - r[i];
            }
            first += nt[i];
        }
        const uint64_t mask = __ballot(g >= 0);
        if (mask) {
            const int src = __builtin_ctzll(mask);
            const uint32_t j = (uint32_t)__builtin_amdgcn_readlane((int)at, src);
            g_out = __builtin_amdgcn_readlane(g, src);
            row0 = (int64_t)__builtin_amdgcn_readlane(base, src) + (int64_t)TM * j;
            rows = min(TM, __builtin_amdgcn_readlane(m, src) - TM * (int)j);
            return true;
        }
        run += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
    }
    return false;
}

// Position -> (token tile, feature tile): groups of GM token tiles, every feature tile of a
// group before the next group, the group's token tiles innermost, so that neighbours share a
// few operand tiles of each kind.
constexpr uint32_t kGroupM = 4;

// Workgroup -> position in that order for the forward expert GEMM's fast kernel.  Workgroups
// are dealt round-robin over the 8 XCDs; XCD x takes tile groups x, x + 8, x + 16, ... (a group is
// kGroupM token tiles across all feature tiles), so that an XCD's workgroups share a
// group's operand tiles in its L2 while the eight XCDs work on neighbouring groups, that
// is on the same expert's weights at the same time.  The remainder past the last whole
// round of 8 groups keeps its order.
__device__ __forceinline__ uint32_t group_interleave(uint32_t bid, uint32_t nblocks, uint32_t gsz)
{
    const uint32_t round = 8 * gsz;
    const uint32_t full = nblocks / round * round;
    if (bid >= full)
        return bid;
    const uint32_t x = bid & 7, slot = bid >> 3;
    return (x + 8 * (slot / gsz)) * gsz + slot % gsz;
}
template <uint32_t GM = kGroupM>
__device__ __forceinline__ void tile_of(uint32_t lin, uint32_t nblocks, uint32_t ntn, uint32_t& mtile,
                                        uint32_t& ntile)
{
    const uint32_t ntm = nblocks / ntn;
    const uint32_t grp = lin / (GM * ntn);
    const uint32_t gm = min(GM, ntm - grp * GM);
    const uint32_t idx = lin - grp * GM * ntn;
    mtile = grp * GM + idx % gm;
    ntile = idx / gm;
}

}  // namespace mxfp4
