// tile_count.h -- how many workgroups a grouped product can need (host code, also for a build
// without a GPU's compiler).
#pragma once

#include <stdint.h>

namespace mxfp4 {

constexpr int kBK = 128;                          // K per stage: one scale block

// Workgroups of TM x TN tiles that a call can need: m rows make at most (m + TM - 1) / TM
// token tiles, and at most min(G, M_cap) experts have rows.
inline int64_t tiles(int64_t M_cap, int32_t G, int64_t N, int TM, int TN)
{
    const int64_t live = G < M_cap ? G : M_cap;
    return (M_cap + live * (TM - 1)) / TM * ((N + TN - 1) / TN);
}

}  // namespace mxfp4
