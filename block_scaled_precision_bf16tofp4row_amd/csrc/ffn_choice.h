// ffn_choice.h -- which kernel of block_ffn.hip a call launches, and in what order its tiles go:
// rules on the sizes alone (host code, also for a build without a GPU's compiler: the tests ask
// it which kernel a size reaches).
#pragma once

#include <math.h>

#include "tile_count.h"

namespace mxfp4 {

enum Kind { kGated, kGradient, kDense };

// The kernels of a call: rows_kernel with 16 or 32 tokens, and the tile kernel of TM tokens x TN
// rows of the weights.  "Split" ones have groups of waves that share K; "Pair" ones fit a CU
// twice and have no groups; the others have a CU for themselves.
enum Which { kRows16, kRows32, k32x64Split, k32x128Split, k32x128Pair, k32x256, k64x64Split, k64x128Split, k128x128Split,
             k128x128Pair, k128x256, k256x256, kKernels };

// What a kernel's workgroup costs: us per block of K, and for its beginning and end.  A CU with
// one workgroup loads 60-78 GB/s whatever the tile, so a block costs by the rows loaded, until
// the matrix instructions count (256 x 256); two workgroups a CU load less each.  Fitted to the
// times of all kernels at 2100 sizes over 1 to 16000 rows of 1 to 32 experts, 16 to 7168
// features and 16 to 7680 deep: the chosen kernel takes 1.03 times the best one's time in the
// mean, 1.11 at most at nine sizes of ten, 1.6 at the worst.
struct Cost {
    int TM, TN;
    bool pair;
    float block, ends;
};
constexpr Cost kCost[kKernels] = {
    {16, 32, false, 0.097f, 2.8f},  {32, 32, false, 0.110f, 2.8f},  {32, 64, false, 0.157f, 3.0f},
    {32, 128, false, 0.290f, 1.9f}, {32, 128, true, 0.360f, 0.45f}, {32, 256, false, 0.540f, 2.2f},
    {64, 64, false, 0.230f, 2.3f},  {64, 128, false, 0.365f, 2.6f}, {128, 128, false, 0.505f, 3.3f},
    {128, 128, true, 0.680f, 1.2f}, {128, 256, false, 0.830f, 4.5f}, {256, 256, false, 1.550f, 5.8f}};
constexpr double kBytesUs = 1 / 10.5e6;           // us a byte of weights
constexpr int64_t kMaxSums = 16 << 20;            // bytes of FP32 sums that are worth a second launch

// Whether a kernel's tiles have whole scale blocks of an E4M3 output.
constexpr bool whole_blocks(Kind kind, Which w) { return kCost[w].TN >= (kind == kGated ? 256 : 128); }

// The kernel of a call, by its estimated time.  fp8: E4M3 outputs are wanted.  The rows are taken
// to be M_cap, the only count that the host has, over all experts.
inline Which choose(Kind kind, bool fp8, int32_t G, int64_t M_cap, int64_t N, int64_t K)
{
    const double n = kind == kGated ? 2.0 * N : N, blocks = (double)((K + kBK - 1) / kBK);
    const double live = (double)(G < M_cap ? G : M_cap);
    const int64_t sums = 4 * M_cap * (kind == kGradient ? 2 * N : N);
    Which best = k256x256;
    double least = INFINITY;
    for (int i = 0; i < kKernels; ++i) {
        const Which w = (Which)i;
        const Cost& c = kCost[i];
        const bool whole = whole_blocks(kind, w);
        if ((kind != kGated || !fp8) && (w == k32x256 || w == k128x256))
            continue;                             // (there for whole scale blocks alone; not timed elsewhere)
        if (fp8 && !whole && sums > kMaxSums)
            continue;
        // an expert's last tile is half full on average, and every expert has one
        const double per = M_cap / (double)c.TM;
        const double each = live > 1 ? fmax(per / live + 0.5, 1) : ceil(per);
        const double wide = ceil(n / c.TN), t = each * live * wide / 256;
        double rounds = ceil(t), block = c.block;
        if (w == k256x256) {
            rounds = fmax(1, t + 0.27 * (ceil(t) - t));        // (partial tiles come last)
            if (t < 1)                            // free CUs leave the others more of the caches and of the clock
                block *= 0.88f + 0.12f * t;
            if (M_cap <= 128 * live)              // tiles of half the size
                block *= 0.57f;
        } else if (c.pair) {
            // past 256 workgroups, empty ones among them, some CUs have two and others none
            rounds = fmax(t, tiles(M_cap, G, (int64_t)n, c.TM, c.TN) > 256 ? 1.4 : 1);
        } else if (live > 1) {
            // the number of tiles is off by the last ones' parts: whether it is past a whole round
            // is a matter of chance
            const double off = sqrt(live / 12) * wide / 256, near = fmax(1, nearbyint(t));
            rounds = fmax(1, near + 0.5 * erfc((near - t) / off * M_SQRT1_2));
        }
        double us = rounds * (blocks * block + c.ends);
        // (the weights' bytes, which reach two XCDs where an expert has more tiles of rows than one)
        us = fmax(us, live * n * K * fmin(each, 2) * kBytesUs);
        if (fp8 && !whole)
            us += 4 + sums * 0.5e-6;              // (the second launch)
        if (us < least) {
            best = w;
            least = us;
        }
    }
    return best;
}

// Whether a tile kernel's tiles go in runs of feature tiles. Pairs of token tiles read the
// weights on two XCDs and the rows on four, runs of feature tiles the weights on one and the
// rows on eight.  So runs, where the weights are most of the bytes and an expert has more than a
// tile of rows: on average over 194 such sizes 0.92 of the pairs' time (330 rows over 6 experts
// x 5376 x 3584 23.2 us, pairs 35.2; 1044 over 10, gradient, x 768 x 4864 16.5, 24.8), at worst
// 1.4 (826 over 22, gradient, x 752 x 2416 23.6, 16.5).  With a tile or less there is nothing to
// share, and pairs spread an expert over all XCDs: 197 rows over 5 experts x 4736 x 2432 14.4
// us, runs 21.8.
inline bool feature_runs(int parts, int TM, int32_t G, int64_t M_cap, int64_t N)
{
    const int64_t live = G < M_cap ? G : M_cap;
    return TM < 256 && live * parts * N > 4 * M_cap && (live > 1 ? 10 * M_cap > 11 * live * TM : M_cap > TM);
}

}  // namespace mxfp4
