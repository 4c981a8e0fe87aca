// block_ffn.hip -- the expert-grouped FP8 product with FP32 block scales (block_tile.h) with
// what a feed-forward layer does to its sums in the same kernel.
//
// With p = A W_g^T (the sums of block_gemm.hip, FP32, not rounded), g the row's expert:
//   gated:     W_g = [Wg; Wu], h = [hg, hu] = p + bias_g, out = act(hg) hu.  A tile has the same
//              features of both halves, so out needs no other workgroup.
//   gradient:  p the gradient of out (A the gradient behind the down projection, W its
//              transpose), h read back: dh = [p hu act'(hg), p act(hg)], and out again.
//   dense:     y = act(p + bias_g) + residual.
// Results leave as BF16, rounded once, or (gated, gradient) as E4M3 rows with an FP32 scale per
// 1x128 block, made from the FP32 values, where the product that follows takes them.
//
// The sums go through LDS as FP32, a tile's rows in one phase or two: a thread then has eight
// consecutive features of a row, 16 lanes a scale block, and its loads and stores are 16 bytes
// in whole lines.
//
// What bounds it: with many rows the product, as in block_gemm.hip (the loads into LDS, then
// power), and the way out of each tile, which only the gradient's makes much of; with few rows
// the weights' bytes; with few rows of few experts the load rate of a CU and, in a program without
// a graph, the host's work per call.
#include <math.h>

#include <algorithm>

#include "activation.h"
#include "block_tile.h"
#include "ffn_choice.h"

namespace mxfp4 {

// What a call reads and writes besides the product's operands.  NULL: not wanted.
struct Ffn {
    const float* bias;                            // [G, C]; C = 2 N (gated), N (dense)
    const uint16_t* h;                            // gradient: [M, 2 N].  dense: the residual [M, N]
    uint16_t* rows;                               // gated: h [M, 2 N].  gradient: dh [M, 2 N].  dense: y [M, N]
    uint16_t* out;                                // gated, gradient: out [M, N].  dense: p + bias [M, N]
    uint8_t* q;                                   // E4M3 of out (gated), of dh (gradient)
    float* q_scales;
    float* sums;                                  // those values in FP32 (where a tile has no whole scale blocks)
    int act;
};

// The epilogue of one thread: eight features, col .. col + 7, of rows of a tile.
template <Kind KIND>
struct Epilogue {
    static constexpr int kParts = KIND == kGated ? 2 : 1;
    // Values of a row in `rows` and in q, per feature.
    static constexpr int kWide = KIND == kDense ? 1 : 2, kQuant = KIND == kGradient ? 2 : 1;
    struct In {
        u32x4 h[2];
    };

    const Ffn& f;
    const uint32_t N;
    const uint32_t col;                           // of a part, in [0, N) or past it
    const bool there;
    __amdgpu_buffer_rsrc_t rh, rrows, rout, rq, rqs, rsums;
    float bias[kParts][8];

    __device__ __forceinline__ Epilogue(const Ffn& f_, const TileAt& at, uint32_t N_, uint32_t c)
        : f(f_), N(N_), col((uint32_t)at.n0 + 8 * c), there((int)(8 * c) < at.cols)
    {
        const uint64_t row = (uint64_t)at.rows;
        if (KIND == kGradient || (KIND == kDense && f.h))
            rh = strip_rsrc(f.h + at.row0 * kWide * N, row * kWide * N * 2);
        if (f.rows)
            rrows = strip_rsrc(f.rows + at.row0 * kWide * N, row * kWide * N * 2);
        if (f.out)
            rout = strip_rsrc(f.out + at.row0 * N, row * N * 2);
        if (KIND != kDense && f.q) {
            rq = strip_rsrc(f.q + at.row0 * kQuant * N, row * kQuant * N);
            rqs = strip_rsrc(f.q_scales + at.row0 * blocks(), row * blocks() * 4);
        }
        if (KIND != kDense && f.sums)
            rsums = strip_rsrc(f.sums + at.row0 * kQuant * N, row * kQuant * N * 4);
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                bias[p][i] = 0.0f;
        if (KIND != kGradient && f.bias && there) {
            const float* const from = f.bias + ((int64_t)at.g * kParts) * N + col;
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const f32x4 b = *reinterpret_cast<const f32x4*>(from + p * (int64_t)N + 4 * j);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        bias[p][4 * j + e] = b[e];
                }
        }
    }
    __device__ __forceinline__ uint32_t blocks() const { return (kQuant * N + 127) / 128; }

    // The byte offset of the thread's features of part p in a row of `wide` parts of elements of
    // `size` bytes; out of range where there are none.
    __device__ __forceinline__ int at_byte(uint32_t row, int wide, int p, int size) const
    {
        return there ? (int)((row * wide * N + p * N + col) * size) : (int)kOutOfRange;
    }
    // What the row needs of memory.
    __device__ __forceinline__ void fetch(uint32_t row, In& in) const
    {
        if constexpr (KIND == kGradient) {
#pragma unroll
            for (int p = 0; p < 2; ++p)
                in.h[p] = __builtin_amdgcn_raw_buffer_load_b128(rh, at_byte(row, 2, p, 2), 0, 2);      // (past the caches)
        } else if constexpr (KIND == kDense) {
            if (f.h)
                in.h[0] = __builtin_amdgcn_raw_buffer_load_b128(rh, at_byte(row, 1, 0, 2), 0, 0);
        }
    }
    static __device__ __forceinline__ void put(__amdgpu_buffer_rsrc_t r, int off, u32x4 v)
    {
        __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 2);      // (past the caches)
    }
    // E4M3 bytes (kBlocks: the 16 lanes of a scale block take part), or FP32 sums.
    template <bool kBlocks>
    __device__ __forceinline__ void quantized(uint32_t row, int p, const float (&v)[8]) const
    {
        if constexpr (kBlocks) {
            if (f.q) {
                float scale;
                const u32x2 b = to_fp8(v, scale);
                __builtin_amdgcn_raw_buffer_store_b64(b, rq, at_byte(row, kQuant, p, 1), 0, 0);
                const uint32_t s = (row * blocks() + (p * N + col) / 128) * 4;
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(scale), rqs,
                                                      there && col % 128 == 0 ? (int)s : (int)kOutOfRange, 0, 0);
            }
        } else if (f.sums) {
            const int off = at_byte(row, kQuant, p, 4);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x4 s = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
                put(rsums, off + 16 * i, __builtin_bit_cast(u32x4, s));
            }
        }
    }
    // Row `row` of the tile: the sums of each part's eight features.
    template <bool kBlocks>
    __device__ __forceinline__ void apply(uint32_t row, float (&v)[kParts][8], const In& in) const
    {
        float slope[8];
        if constexpr (KIND != kGradient) {
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[p][i] += bias[p][i];
        }
        if constexpr (KIND == kGated) {
            if (f.rows) {
                put(rrows, at_byte(row, 2, 0, 2), to_bf16(v[0]));
                put(rrows, at_byte(row, 2, 1, 2), to_bf16(v[1]));
            }
            activate8<false>(f.act, v[0], slope);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[0][i] *= v[1][i];
            if (f.out)
                put(rout, at_byte(row, 1, 0, 2), to_bf16(v[0]));
            quantized<kBlocks>(row, 0, v[0]);
        } else if constexpr (KIND == kGradient) {
            float a[8], u[8];
            from_bf16(in.h[0], a);
            from_bf16(in.h[1], u);
            activate8<true>(f.act, a, slope);
            float dg[8], du[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dg[i] = v[0][i] * u[i] * slope[i];
                du[i] = v[0][i] * a[i];
                u[i] *= a[i];
            }
            if (f.out)
                put(rout, at_byte(row, 1, 0, 2), to_bf16(u));
            if (f.rows) {
                put(rrows, at_byte(row, 2, 0, 2), to_bf16(dg));
                put(rrows, at_byte(row, 2, 1, 2), to_bf16(du));
            }
            quantized<kBlocks>(row, 0, dg);
            quantized<kBlocks>(row, 1, du);
        } else {
            if (f.out)
                put(rout, at_byte(row, 1, 0, 2), to_bf16(v[0]));
            activate8<false>(f.act, v[0], slope);
            if (f.h) {
                from_bf16(in.h[0], slope);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[0][i] += slope[i];
            }
            put(rrows, at_byte(row, 1, 0, 2), to_bf16(v[0]));
        }
    }
};

// A tile's way out: its sums through LDS to the epilogue.
template <class W, Kind KIND>
__device__ __forceinline__ void tile_out(uint8_t* lds0, uint8_t* lds1, uint8_t* lds2, uint8_t* lds3,
                                         const typename W::State& t, const Ffn& f, const TileAt& at, int64_t N)
{
    constexpr int kParts = Epilogue<KIND>::kParts;
    constexpr int WM = W::kWM, MT = W::kMT, NT = W::kNT, TM = W::TM, TN = W::TN, kThreads = W::kThreads;
    // Groups of 16 rows, those of wave row wm one after the other; kGroups of them fit the LDS.
    constexpr int kGroup = 16 * TN * 4, kIn0 = W::kBuf / kGroup, kIn2 = W::kBuf2 / kGroup, kIn3 = W::kBuf3 / kGroup;
    constexpr int kGroups = 2 * kIn0 + kIn2 + kIn3, kPhases = TM / 16 <= kGroups ? 1 : 2;
    constexpr int MP = MT / kPhases, kRows = TM / kPhases;
    static_assert(kIn0 >= 1 && kRows / 16 <= kGroups && MT % kPhases == 0, "a phase's rows fit the LDS");
    auto place = [&](int group, int q) {           // (q: the group of waves whose sums they are)
        return group < kIn0             ? lds0 + q * W::kBuf + group * kGroup
               : group < 2 * kIn0        ? lds1 + q * W::kBuf + (group - kIn0) * kGroup
               : group < 2 * kIn0 + kIn2 ? lds2 + q * W::kBuf2 + (group - 2 * kIn0) * kGroup
                                         : lds3 + q * W::kBuf3 + (group - 2 * kIn0 - kIn2) * kGroup;
    };
    // 16-byte chunk c of row r is at chunk c ^ (r % 16).
    auto chunk_at = [](uint32_t ch, uint32_t row) { return 16 * (ch ^ row); };
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) % W::kWaves;
    const int mine = W::kSplit == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 6) / W::kWaves;
    const int wm = wave % WM, wn = wave / WM;
    const uint32_t r = (uint32_t)(tid & 15), h = (uint32_t)(tid >> 4 & 3);
    // threads of a row, and rows of a step; threads past kWork have nothing to do
    constexpr int kCols = TN / kParts / 8, kWork = kThreads < kRows * kCols ? kThreads : kRows * kCols;
    constexpr int kStep = kWork / kCols;
    static_assert(kWork % 64 == 0 && kRows % kStep == 0 && kStep % (64 / kCols) == 0 && 64 % kCols == 0, "rows");
    const uint32_t c = (uint32_t)tid % kCols;
    typedef Epilogue<KIND> E;
    const E epi(f, at, (uint32_t)N, c);
    // A batch's rows are fetched while the one before it is worked on.
    constexpr int kSteps = kRows / kStep, kBatch = kSteps < 4 ? kSteps : 4, kBatches = kPhases * kSteps / kBatch;
    static_assert(kSteps % kBatch == 0, "whole batches");
    auto write = [&](auto p) {
        constexpr int kPhase = decltype(p)::value;
#pragma unroll
        for (int m = 0; m < MP; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                *reinterpret_cast<f32x4*>(place(wm * MP + m, mine) + r * (TN * 4) +
                                          chunk_at((uint32_t)(4 * (NT * wn + nt)) + h, r)) =
                    t.acc[kPhase * MP + m][nt];
            }
        // (keeps the compiler from merging the phases' code, with pointers into the sums)
        asm volatile("; phase %0" ::"n"(kPhase));
    };
    // (rows of a phase: group by group; step i of all is row `in` of phase i / kSteps, which is
    // this row of the tile)
    auto row_of = [&](int i) {
        const uint32_t in = (uint32_t)tid / kCols + kStep * (i % kSteps), group = in / 16;
        return 16 * (MT * (group / MP) + i / kSteps * MP + group % MP) + in % 16;
    };
    typename E::In in[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
        epi.fetch(row_of(u), in[u]);
#pragma unroll 1
    for (int b = 0; b < kBatches; ++b) {
        if (b % (kSteps / kBatch) == 0) {
            if (b == 0) {
                write(std::integral_constant<int, 0>{});
            } else {
                meet();                           // the rows of the phase before have been read
                write(std::integral_constant<int, kPhases - 1>{});
            }
            meet();
        }
        if (kWork < kThreads && tid >= kWork)
            continue;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = b * kBatch + u;
            const uint32_t at_row = (uint32_t)tid / kCols + kStep * (i % kSteps), rr = at_row % 16;
            const int group = __builtin_amdgcn_readfirstlane((int)(at_row / 16));
            float v[kParts][8];
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t from = rr * (TN * 4) + chunk_at(p * (TN / 8) + 2 * c + j, rr);
                    f32x4 s = *reinterpret_cast<const f32x4*>(place(group, 0) + from);
#pragma unroll
                    for (int q = 1; q < W::kSplit; ++q)
                        s += *reinterpret_cast<const f32x4*>(place(group, q) + from);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[p][4 * j + e] = s[e];
                }
            epi.template apply<TN / kParts % 128 == 0>(row_of(i), v, in[u]);
            if (b + 1 < kBatches)
                epi.fetch(row_of(i + kBatch), in[u]);
        }
    }
}

// The large tile, 256 x 256 with 8 waves, in us (8 experts, SiLU; the operations alone at the
// 3.25 PFLOP/s of a large product without block scales):
//   gated, 16384 rows x 2048 x 7168, BF16 out and h: 481-501 (296)
//   gradient of it, dh and out:                       295-308 (148; matrix units 36 % busy, gated 47 %)
//   dense, 8192 rows x 4096 x 7168, GELU, p kept:     225-261, one expert (148)
// A CU has one such workgroup.  So a last round that a part of the tiles needs costs nearly a
// whole one: the same rows in equal shares, two rounds and four, take 254-258 and 449.  And
// nothing hides the gradient's way out, about 11 us of vector work a tile and 134 MB of h.
// Fetching h's lines during the last stages cost more than it hid (342 -> 355 us, with an earlier
// form of both).
// Few rows an expert, 32 a tile, read the weights at 5.7-6 TB/s: 128 rows over 32 experts
// x 2048 x 7168 gated with FP8 out 155, 940 MB; dense x 7168 x 2048 80, 470 MB.
template <class W, Kind KIND>
__global__ __launch_bounds__(W::kThreads, W::kD == 2 && W::kSplit == 1 ? 2 : 1) void ffn_tile_kernel(
    const uint8_t* __restrict__ a, const float* __restrict__ sa, const uint8_t* __restrict__ w,
    const float* __restrict__ sw, Ffn f, const int32_t* __restrict__ offs, int G, int64_t N, int64_t K, uint32_t ntn,
    bool by_feature)
{
    constexpr int kParts = Epilogue<KIND>::kParts;
    // separate arrays: what is loaded into one does not hold up reads of another
    __shared__ __attribute__((aligned(16))) uint8_t lds0[W::kSplit * W::kBuf];
    __shared__ __attribute__((aligned(16))) uint8_t lds1[W::kSplit * W::kBuf];
    __shared__ __attribute__((aligned(16))) uint8_t lds2[W::kSplit * W::kBuf2];
    __shared__ __attribute__((aligned(16))) uint8_t lds3[W::kSplit * W::kBuf3];
    TileAt at;
    if (!tile_place<W::TM, W::TN, kParts, W::TM == 256>(offs, G, N, ntn, at, by_feature))
        return;                                   // uniform over the workgroup
    auto tile = [&](auto type) {
        typedef decltype(type) T;
        typename T::State t;
        tile_sums<T, kParts>(lds0, lds1, lds2, lds3, a, sa, w, sw, N, K, at, t);
        tile_out<T, KIND>(lds0, lds1, lds2, lds3, t, f, at, N);
    };
    if constexpr (W::TM == 256) {
        // half a tile's rows or fewer: a tile of half the size
        typedef Tile<2, 4, 4, 4, 2> Half;
        static_assert(Half::kBuf <= W::kBuf && Half::kBuf2 <= W::kBuf2 && Half::kBuf3 <= W::kBuf3, "the same LDS");
        if (at.rows > Half::TM)
            tile(W{});
        else
            tile(Half{});
    } else {
        tile(W{});
    }
}

// One expert's 16 or 32 rows and 32 rows of the weights a workgroup, whose waves share K: one row
// x 2048 x 7168 gated 9.0 us (29 MB of weights, 3.3 TB/s: what 128 of 256 CUs load), dense 7168 x
// 2048 with a residual 5.5.
template <int MT, Kind KIND>
__global__ __launch_bounds__(64 * kRowsWaves) void ffn_rows_kernel(
    const uint8_t* __restrict__ a, const float* __restrict__ sa, const uint8_t* __restrict__ w,
    const float* __restrict__ sw, Ffn f, const int32_t* __restrict__ offs, int G, int64_t N, int64_t K, uint32_t ntm)
{
    typedef RowsTile<MT> R;
    typedef Epilogue<KIND> E;
    constexpr int kParts = E::kParts;
    // separate arrays: what is loaded into one does not hold up reads of another
    __shared__ __attribute__((aligned(16))) uint8_t lds0[kRowsWaves * R::kBuf];
    __shared__ __attribute__((aligned(16))) uint8_t lds1[kRowsWaves * R::kBuf];
    __shared__ __attribute__((aligned(16))) uint8_t lds2[kRowsWaves * R::kBuf];
    __shared__ __attribute__((aligned(16))) uint8_t lds3[kRowsWaves * R::kBuf];
    __shared__ __attribute__((aligned(16))) typename R::Part part[kRowsWaves];
    TileAt at;
    if (!rows_place<R::TM, kParts>(offs, G, N, ntm, at))
        return;                                   // uniform over the workgroup
    constexpr int kCols = R::TN / kParts / 8;
    static_assert(R::TM * kCols <= 64 * kRowsWaves, "one item a thread");
    const uint32_t row = threadIdx.x / kCols, c = threadIdx.x % kCols;
    // what the epilogue reads is on its way before the product's loads (the loop's counted
    // waits then wait for it too, never for less)
    const E epi(f, at, (uint32_t)N, c);
    typename E::In in;
    epi.fetch(row, in);
    rows_sums<MT, kParts>(lds0, lds1, lds2, lds3, part, a, sa, w, sw, N, K, at);
    if (row >= R::TM)
        return;
    float v[kParts][8];
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f32x4 s = R::sum(part, row, p * (R::TN / 2) + 8 * c + 4 * j);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[p][4 * j + e] = s[e];
        }
    epi.template apply<false>(row, v, in);
}

// FP32 rows [0, offs[G]) of `cols` values -> E4M3 rows with FP32 scales: 16 lanes of eight
// values to a block, blocks of a row one after the other.  2 us for a row of 2048.  (The tiles of
// few rows are narrower than a block; joining their maxima in one launch would take counters that
// every call has to find cleared.)
__global__ __launch_bounds__(kThreads) void quantize_sums_kernel(
    const float* __restrict__ x, uint8_t* __restrict__ q, float* __restrict__ q_scales,
    const int32_t* __restrict__ offs, int G, uint32_t cols, uint32_t blocks)
{
    const uint64_t block = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / 16;
    const int64_t row = (int64_t)(block / blocks);
    const uint32_t b = (uint32_t)(block % blocks), col = 128 * b + 8 * (threadIdx.x % 16);
    if (row >= offs[G])
        return;                                   // (16 lanes leave together)
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (col < cols) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f32x4 s = *reinterpret_cast<const f32x4*>(x + row * cols + col + 4 * j);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[4 * j + e] = s[e];
        }
    }
    float scale;
    const u32x2 bytes = to_fp8(v, scale);
    if (col < cols)
        *reinterpret_cast<u32x2*>(q + row * cols + col) = bytes;
    if (threadIdx.x % 16 == 0)
        q_scales[row * blocks + b] = scale;
}

namespace {

typedef Tile<1, 2, 2, 2, 3, 4> T32x64Split;
typedef Tile<1, 4, 2, 2, 3, 2> T32x128Split;
typedef Tile<1, 4, 2, 2, 3> T32x128Pair;
typedef Tile<1, 4, 2, 4, 4> T32x256;
typedef Tile<2, 2, 2, 2, 4, 2> T64x64Split;
typedef Tile<1, 4, 4, 2, 3, 2> T64x128Split;
typedef Tile<2, 2, 4, 4, 2, 2> T128x128Split;
typedef Tile<2, 2, 4, 4, 2> T128x128Pair;
typedef Tile<2, 4, 4, 4, 3> T128x256;
typedef Tile<2, 4, 8, 4, 2> T256x256;

template <class T>
constexpr bool is(Which w) { return kCost[w].TM == T::TM && kCost[w].TN == T::TN; }
static_assert(is<T32x64Split>(k32x64Split) && is<T32x128Split>(k32x128Split) && is<T32x128Pair>(k32x128Pair) &&
              is<T32x256>(k32x256) && is<T64x64Split>(k64x64Split) && is<T64x128Split>(k64x128Split) &&
              is<T128x128Split>(k128x128Split) && is<T128x128Pair>(k128x128Pair) && is<T128x256>(k128x256) &&
              is<T256x256>(k256x256), "the sizes that the choice goes by");

template <Kind KIND>
hipError_t launch_ffn(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, Ffn f,
                      const int32_t* offs, int32_t G, int64_t M_cap, int64_t N, int64_t K, hipStream_t stream)
{
    constexpr int kParts = Epilogue<KIND>::kParts;
    const Which which = choose(KIND, f.q != nullptr, G, M_cap, N, K);
    const bool then = f.q && !whole_blocks(KIND, which);
    int g = G;
    int64_t n = N, k = K;
    uint32_t nt = 0;                              // feature tiles (tile kernel), token tiles (rows kernel)
    bool by_feature = false;                      // (tile kernel)
    void* args[] = {(void*)&a, (void*)&sa, (void*)&w, (void*)&sw, (void*)&f, (void*)&offs, (void*)&g,
                    (void*)&n, (void*)&k, (void*)&nt, (void*)&by_feature};
    auto launch = [&](const void* kernel, int64_t grid, int threads) {
        return grid > 0x7FFFFFFF ? hipErrorInvalidValue
                                 : launch_kernel(kernel, dim3((unsigned)grid), dim3((unsigned)threads), args, stream, !then);
    };
    auto tile = [&](auto type) {
        typedef decltype(type) T;
        nt = (uint32_t)((N + T::TN / kParts - 1) / (T::TN / kParts));
        by_feature = feature_runs(kParts, T::TM, G, M_cap, N);
        return launch((const void*)ffn_tile_kernel<T, KIND>, tiles(M_cap, G, N, T::TM, T::TN / kParts), T::kThreads);
    };
    auto rows = [&](int TM, const void* kernel) {
        nt = (uint32_t)tiles(M_cap, G, 1, TM, 1);
        return launch(kernel, tiles(M_cap, G, N, TM, kRowsTN / kParts), 64 * kRowsWaves);
    };
    auto first = [&]() {
        switch (which) {
        case kRows16: return rows(16, (const void*)ffn_rows_kernel<1, KIND>);
        case kRows32: return rows(32, (const void*)ffn_rows_kernel<2, KIND>);
        case k32x64Split: return tile(T32x64Split{});
        case k32x128Split: return tile(T32x128Split{});
        case k32x128Pair: return tile(T32x128Pair{});
        case k64x64Split: return tile(T64x64Split{});
        case k64x128Split: return tile(T64x128Split{});
        case k128x128Split: return tile(T128x128Split{});
        case k128x128Pair: return tile(T128x128Pair{});
        case k256x256: return tile(T256x256{});
        default: break;
        }
        if constexpr (KIND == kGated)
            return which == k32x256 ? tile(T32x256{}) : tile(T128x256{});
        return hipErrorInvalidValue;              // (no other kind chooses these)
    };
    const hipError_t e = first();
    if (e != hipSuccess || !then)
        return e;
    uint32_t cols = (uint32_t)(Epilogue<KIND>::kQuant * N), blocks = (cols + 127) / 128;
    void* more[] = {(void*)&f.sums, (void*)&f.q, (void*)&f.q_scales, (void*)&offs, (void*)&g, (void*)&cols,
                    (void*)&blocks};
    const int64_t groups = (M_cap * blocks * 16 + kThreads - 1) / kThreads;
    return groups > 0x7FFFFFFF ? hipErrorInvalidValue
                               : launch_kernel((const void*)quantize_sums_kernel, dim3((unsigned)groups),
                                               dim3(kThreads), more, stream);
}

}  // namespace

// Whether a call with E4M3 outputs uses its workspace, and the bytes that it and every call of
// fewer rows use at most.
bool gated_uses_workspace(int32_t G, int64_t M_cap, int64_t I, int64_t K)
{
    return !whole_blocks(kGated, choose(kGated, true, G, M_cap, I, K));
}
bool gated_backward_uses_workspace(int32_t G, int64_t M_cap, int64_t I, int64_t K)
{
    return !whole_blocks(kGradient, choose(kGradient, true, G, M_cap, I, K));
}
int64_t gated_workspace(int64_t M_cap, int64_t I) { return std::min(4 * M_cap * I, kMaxSums); }
int64_t gated_backward_workspace(int64_t M_cap, int64_t I) { return std::min(8 * M_cap * I, kMaxSums); }

hipError_t launch_gated_gemm(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, const float* bias,
                             uint16_t* out, uint8_t* q, float* q_scales, uint16_t* h, float* work,
                             const int32_t* offs, int32_t G, int64_t M_cap, int64_t I, int64_t K, int act,
                             hipStream_t stream)
{
    const Ffn f = {bias, nullptr, h, out, q, q_scales, q ? work : nullptr, act};
    return launch_ffn<kGated>(a, sa, w, sw, f, offs, G, M_cap, I, K, stream);
}

hipError_t launch_gated_gemm_backward(const uint8_t* dy, const float* sdy, const uint8_t* wt, const float* swt,
                                      const uint16_t* h, uint16_t* dh, uint8_t* q, float* q_scales, uint16_t* out,
                                      float* work, const int32_t* offs, int32_t G, int64_t M_cap, int64_t I,
                                      int64_t K, int act, hipStream_t stream)
{
    const Ffn f = {nullptr, h, dh, out, q, q_scales, q ? work : nullptr, act};
    return launch_ffn<kGradient>(dy, sdy, wt, swt, f, offs, G, M_cap, I, K, stream);
}

hipError_t launch_block_gemm_act(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw,
                                 const float* bias, const uint16_t* residual, uint16_t* pre, uint16_t* y,
                                 const int32_t* offs, int32_t G, int64_t M_cap, int64_t N, int64_t K, int act,
                                 hipStream_t stream)
{
    const Ffn f = {bias, residual, y, pre, nullptr, nullptr, nullptr, act};
    return launch_ffn<kDense>(a, sa, w, sw, f, offs, G, M_cap, N, K, stream);
}

}  // namespace mxfp4
