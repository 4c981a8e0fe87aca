// tiles.h -- the expert GEMMs' map from workgroups to (expert, token tile, feature tile).
#pragma once

#include "strips.h"

namespace mxfp4 {

// Token tile `mtile` (tiles of TM rows, in expert order) -> expert, its first row and the
// tile's rows.
// False if the tile does not exist.  Experts are scanned 64 at a time, one per lane.
template <int TM>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ offs, int G, uint32_t mtile,
                                          int& g_out, int64_t& row0, int& rows)
{
    const int lane = threadIdx.x & 63;
    uint32_t run = 0;
    for (int g0 = 0; g0 < G; g0 += 64) {
        const int h = g0 + lane;
        const int32_t r0 = h < G ? offs[h] : 0;
        const int32_t mg = h < G ? offs[h + 1] - r0 : 0;
        const uint32_t nt = (uint32_t)(mg + TM - 1) / TM;
        uint32_t incl = nt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = __shfl_up(incl, d, 64);
            if (lane >= d)
                incl += o;
        }
        const uint32_t first = run + incl - nt;
        const uint64_t mask = __ballot(nt > 0 && mtile >= first && mtile < first + nt);
        if (mask) {
            const int src = __builtin_ctzll(mask);
            const uint32_t j = mtile - (uint32_t)__builtin_amdgcn_readlane((int)first, src);
            const int32_t base = __builtin_amdgcn_readlane(r0, src);
            const int32_t m = __builtin_amdgcn_readlane(mg, src);
            g_out = g0 + src;
            row0 = (int64_t)base + (int64_t)TM * j;
            rows = min(TM, m - TM * (int)j);
            return true;
        }
        run = uniform(run + (uint32_t)__shfl(incl, 63, 64));
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
