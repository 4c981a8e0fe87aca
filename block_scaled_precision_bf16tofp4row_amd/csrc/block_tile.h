// block_tile.h -- the FP8 product with FP32 block scales up to its FP32 sums: the stage loop of
// the tile kernels and the K-splitting loop for few rows, for the kernels that differ in what
// they do with the sums (block_gemm.hip rounds them to BF16, block_ffn.hip has activations,
// biases and gradients behind them).
//
// kParts = 1: a tile's TN rows of the weights are TN consecutive features.  kParts = 2: the
// weights of an expert are two matrices of N features, one after the other ([G, 2, N, K], the
// scales [G, 2, ceil(N/128), ceil(K/128)]), and a tile's first TN / 2 rows are features of the
// first, the others the same features of the second.
#pragma once

#include "tile_count.h"
#include "tiles.h"

namespace mxfp4 {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kOutOfRange = 0x80000000u;     // offset past every buffer's range
// s_waitcnt immediate (gfx9 encoding) that waits for vmcnt <= n and nothing else.
constexpr int vmcnt_at_most(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }
constexpr int kUnitScale = 0x7F7F7F7F;            // E8M0 bytes of 1.0

// Memory to LDS: lane L's 16 (or 4) bytes at offset off + k0 of the resource land at `to` +
// 16 L (4 L).
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t off, uint32_t k0)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) uint8_t*)to, 16, off, (int)k0, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t off)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) uint8_t*)to, 4, off, 0, 0, 0);
}

// A lane's fragment of one operand row for 64 of K: the row's 16-byte LDS chunks at byte
// offsets c0 and c1.
__device__ __forceinline__ i32x8 frag(const uint8_t* rowp, uint32_t c0, uint32_t c1)
{
    const u32x4 v0 = *reinterpret_cast<const u32x4*>(rowp + c0);
    const u32x4 v1 = *reinterpret_cast<const u32x4*>(rowp + c1);
    return i32x8{(int)v0.x, (int)v0.y, (int)v0.z, (int)v0.w, (int)v1.x, (int)v1.y, (int)v1.z, (int)v1.w};
}

__device__ __forceinline__ f32x4 mfma128(i32x8 w, i32x8 a, f32x4 c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 0, 0, 0, kUnitScale, 0, kUnitScale);
}

// A workgroup barrier behind this wave's LDS reads and writes.  __syncthreads would also wait
// for every load into LDS in flight, those of the stages to come among them; the stage loop
// waits for the ones it needs by count.
__device__ __forceinline__ void meet()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// What a wave needs in its stage loop.
template <int D>
struct TileCtx {
    uint8_t* buf[D];                              // the LDS stage buffers
    uint8_t* late[2];                             // with two: the rows of the later half of the tokens
    __amdgpu_buffer_rsrc_t ra, rw, rsa, rsw;      // operand rows, token and weight scales
    uint32_t abase, wbase, ac0, ac1, wc0, wc1, K; // loader: row offsets and the two chunk offsets of each
    uint32_t lds_a, lds_w, lds_s;                 // loader: LDS offsets of the wave's first rows, scale slots
    uint32_t srow, sslot;                         // scale loader: global offset of the row, LDS slot
    uint32_t arow, wrow, c0, c1;                  // fragments: LDS offsets of the lane's rows, chunks
    uint32_t scl_at;                              // slot of the lane's first token scale
    uint32_t turn, blocks;                        // the block of K that stage 0 takes, and their number
    uint32_t first, count;                        // where groups of waves share K: this group's blocks
};

// The tile of WM x WN waves, each 16 MT tokens x 16 NT features, with D stage buffers.  SPLIT > 1:
// so many groups of these waves, each with buffers of its own and a run of K's blocks.
template <int WM, int WN, int MT, int NT, int D, int SPLIT = 1>
struct Tile {
    static constexpr int kWM = WM, kWN = WN, kMT = MT, kNT = NT, kD = D, kSplit = SPLIT;
    static constexpr int TM = 16 * MT * WM, TN = 16 * NT * WN;
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves * SPLIT;      // (of a group; of all)
    static constexpr int kLoadsA = TM / 8 / kWaves, kLoadsW = TN / 8 / kWaves;   // 8-row loads of a wave
    static constexpr int kSlots = 64 * kWaves;              // scale slots (those past TM are not read)
    static constexpr int kTiles = MT * NT;
    // Where rows are a multiple of 4096 bytes apart, a stage's 128-byte pieces of all rows lie
    // in few memory channels.  The tile for few rows, which lives on the weights' stream, then
    // starts each feature tile and expert at another block of K and goes round (64 rows over
    // 128 experts x 4096 x 4096: 138 us, 160 all from the start; at 7168 deep it would cost 5 %).
    static constexpr bool kTurn = TM == 32;
    static constexpr int kLag = 3;                          // products in flight before their scaled add
    static constexpr int kLoads = kLoadsA + kLoadsW + 2;
    // With two buffers, the earlier half of each wave's token tiles, the weights and the scales
    // of a later stage are loaded from the middle of a stage on, as soon as this stage's are in
    // registers; the rest after the stage's barrier, as all of it with more buffers.
    static constexpr bool kHalves = D == 2;
    // A buffer: token rows (the early ones), weights' rows, then a wave's token scales and its
    // weights' scale.
    static constexpr int kTok = kHalves ? TM / 2 : TM;
    static constexpr int kScales = (kTok + TN) * kBK;
    static constexpr int kBuf = kScales + 8 * kSlots;
    static constexpr int kLate = kHalves ? TM / 2 * kBK : 0;
    static constexpr int kEarlyOps = kHalves ? kLoadsW + kLoadsA / 2 : 0;
    // While stage s + 1 is awaited, the loads of later stages may be in flight: s + 2's early
    // ones, or all of s + 2 .. s + D - 1.
    static constexpr int kInFlight = kHalves ? kEarlyOps + 2 : (D - 2) * kLoads;
    static constexpr int kBuf2 = D > 2 ? kBuf : kLate, kBuf3 = D > 3 ? kBuf : kHalves ? kLate : 16;   // lds2, lds3
    static_assert(D >= 2 && D <= 4, "stage buffers");
    static_assert(TM % (8 * kWaves) == 0 && TN % (8 * kWaves) == 0 && TM <= kSlots, "loads");
    static_assert((TN % 128 == 0 || 128 % TN == 0) && 128 % (16 * NT) == 0, "a wave's features lie in one scale block");
    static_assert(!kHalves || (MT % 2 == 0 && kLoadsA % 2 == 0 && MT >= 4), "halves");
    static_assert((MT == 2 || MT % 4 == 0) && kTiles % 4 == 0, "scale reads, ring of products");

    struct State {
        f32x4 acc[MT][NT];
        f32x4 p[4];                               // products on their way to acc
        i32x8 fw[NT], fa[2];
        float raw[MT], sc[MT];                    // next and present token scales (sc: times the weights')
        float wsc[D];                             // the weights' scale of the stages
    };

    static constexpr uint32_t kNoBlock = 0xFFFFFF;          // past K for every K
    // The block of K that stage s takes.
    static __device__ __forceinline__ uint32_t block_of(const TileCtx<D>& cx, uint32_t s)
    {
        if constexpr (SPLIT > 1) {
            const uint32_t in = kTurn ? s + cx.turn < cx.count ? s + cx.turn : s + cx.turn - cx.count : s;
            return s < cx.count ? cx.first + in : kNoBlock;
        }
        if constexpr (!kTurn)
            return s;
        const uint32_t b = s + cx.turn;
        return s < cx.blocks ? b < cx.blocks ? b : b - cx.blocks : cx.blocks;
    }
    // Operand loads `from` .. `to` - 1 of stage s into buffer b = s % D, the weights' first, then
    // the tokens'.  Offsets are made here, from registers that live across the stages; a stage
    // past the last reads nothing (its columns are past K).
    static __device__ __forceinline__ void issue_operands(const TileCtx<D>& cx, int b, uint32_t s, int from, int to)
    {
        // (the resource's range is less than 128 K for an expert of few rows, so a block past the
        // last is given no scalar offset: what is left of the range would be negative)
        const uint32_t kb = block_of(cx, s);
        const bool past = kb >= cx.blocks;
        const uint32_t k0 = past ? 0 : kb * kBK, K = past ? 0 : cx.K;
#pragma unroll
        for (int j = from; j < to; ++j) {
            const bool tok = j >= kLoadsW;
            const int i = tok ? j - kLoadsW : j;
            constexpr int kInHalf = kHalves ? kLoadsA / 2 : kLoadsA + 1;
            const int half = tok ? i / kInHalf : 0, in_half = tok ? i % kInHalf : i;
            const int rows = 8 * (in_half + half * MT);
            uint8_t* const to_buf = half ? cx.late[b] : cx.buf[b];
            const uint32_t c = tok ? (in_half & 1 ? cx.ac1 : cx.ac0) : (i & 1 ? cx.wc1 : cx.wc0);
            const uint32_t off = c + k0 < K ? (tok ? cx.abase : cx.wbase) + c : kOutOfRange;
            load16_to_lds(tok ? cx.ra : cx.rw, to_buf + (tok ? cx.lds_a : cx.lds_w) + 8 * in_half * kBK,
                          off + (uint32_t)rows * cx.K, k0);
        }
    }
    // Its scales.
    static __device__ __forceinline__ void issue_scales(const TileCtx<D>& cx, int b, uint32_t s)
    {
        const uint32_t kb = block_of(cx, s);
        uint8_t* const to = cx.buf[b] + kScales + cx.lds_s;
        load4_to_lds(cx.rsa, to, kb * kBK < cx.K ? cx.srow + 4 * kb : kOutOfRange);
        load4_to_lds(cx.rsw, to + 4 * kSlots, 4 * kb);
    }
    // The scales of stage s (buffer b).
    static __device__ __forceinline__ void read_scales(const TileCtx<D>& cx, State& t, int b)
    {
        const float* const from = reinterpret_cast<const float*>(cx.buf[b] + kScales);
#pragma unroll
        for (int i = 0; i < MT; ++i)
            t.raw[i] = from[cx.scl_at + i];
        t.wsc[b] = from[kSlots + cx.sslot];
    }
    static __device__ __forceinline__ i32x8 token_frag(const TileCtx<D>& cx, int b, int mt)
    {
        const uint8_t* const from = kHalves && mt >= MT / 2 ? cx.late[b] : cx.buf[b];
        return frag(from + cx.arow + 16 * (kHalves ? mt % (MT / 2) : mt) * kBK, cx.c0, cx.c1);
    }
    static __device__ __forceinline__ i32x8 weight_frag(const TileCtx<D>& cx, int b, int nt)
    {
        return frag(cx.buf[b] + cx.wrow + 16 * nt * kBK, cx.c0, cx.c1);
    }
    // The scaled add of product I of a stage (of the stage before, for I < 0).
    template <int I>
    static __device__ __forceinline__ void add(State& t)
    {
        constexpr int i = (I + kTiles) % kTiles, mt = i / NT, nt = i % NT;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            t.acc[mt][nt][e] = __builtin_fmaf(t.sc[mt], t.p[i & 3][e], t.acc[mt][nt][e]);
    }
    // Products I .. END - 1 of the stage in buffer b, each followed by the scaled add of the one
    // kLag before it, in this order (the scheduler would put dependent ones together), and by
    // loads of stage s into this buffer, where they are due.  In the stage's last token tile a
    // weight fragment is replaced by the next stage's after its use.
    template <int I, int END>
    static __device__ __forceinline__ void products(const TileCtx<D>& cx, State& t, int b, uint32_t s)
    {
        if constexpr (I < END) {
            constexpr int mt = I / NT, nt = I % NT, kOps = kLoadsA + kLoadsW;
            t.p[I & 3] = mfma128(t.fw[nt], t.fa[mt % 2], f32x4{});
            if constexpr (mt == MT - 1) {
                t.fw[nt] = weight_frag(cx, (b + 1) % D, nt);
                issue_operands(cx, b, s, kEarlyOps + nt * (kOps - kEarlyOps) / NT,
                               kEarlyOps + (nt + 1) * (kOps - kEarlyOps) / NT);
            } else if constexpr (kHalves && mt == MT / 2) {
                issue_operands(cx, b, s, nt * kEarlyOps / NT, (nt + 1) * kEarlyOps / NT);
            }
            if constexpr (I >= kLag)
                add<I - kLag>(t);
            __builtin_amdgcn_sched_barrier(0);
            products<I + 1, END>(cx, t, b, s);
        }
    }
    template <int M>
    static __device__ __forceinline__ void token_tiles(const TileCtx<D>& cx, State& t, int b, uint32_t s)
    {
        if constexpr (M < MT - 1) {
            if constexpr (kHalves && M == MT / 2) {
                meet();                           // every wave has the weights and half the tokens in registers
                issue_scales(cx, b, s);
            }
            t.fa[(M + 1) % 2] = token_frag(cx, b, M + 1);
            __builtin_amdgcn_sched_barrier(0);
            products<M * NT, (M + 1) * NT>(cx, t, b, s);
            token_tiles<M + 1>(cx, t, b, s);
        }
    }
    // Stage s in buffer B = s % D.
    template <int B>
    static __device__ __forceinline__ void stage(const TileCtx<D>& cx, State& t, uint32_t s)
    {
        constexpr int kNext = (B + 1) % D;
        add<-3>(t);
        add<-2>(t);
        add<-1>(t);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            t.sc[mt] = t.raw[mt] * t.wsc[B];
        token_tiles<0>(cx, t, B, s + D);
        // every fragment of this stage is in registers: wait for the next one's loads, meet
        // the others, and load (the rest of) a later one into this buffer
        __builtin_amdgcn_s_waitcnt(vmcnt_at_most(kInFlight));
        meet();
        t.fa[0] = token_frag(cx, kNext, 0);
        read_scales(cx, t, kNext);
        if constexpr (!kHalves)
            issue_scales(cx, B, s + D);
        products<(MT - 1) * NT, kTiles>(cx, t, B, s + D);
    }
};

// The tile kernels' loop: WM x WN waves, K in stages of 128 (one scale block) through D LDS buffers.
// LDS rows are 128 bytes with 16-byte chunk c of row r at chunk c ^ ((r >> 1) & 7), so that
// the fragment reads of 16 rows hit distinct banks; operand bytes go there straight from
// memory.  A stage: products of all but the last token tile, each token fragment read one
// tile ahead; wait for the next stage's loads, barrier; products of the last token tile,
// while the next stage's first fragments are read (a weight fragment right after its last
// use) and a later stage's loads go out into the buffer just left.  So the barrier never
// finds a wave without matrix work behind it.  The scaled adds run three products late and
// the loads go out one or two at a time between products (256 x 256, 32768 rows x 7168 x
// 4096: 890-940 us; adds two late 925-960; all loads in a burst behind the barrier as well
// 970-990; with zeros for operands, which leave the clock at its top, 784).
// D = 2 for the large tiles, whose buffers fill a CU's LDS or half of it.  A load then has one
// stage to arrive, so most of them go out half a stage earlier, behind a barrier in the
// middle: 8 experts, 2048 rows x 4096 x 7168: 102 us (256 x 256), 119 (128 x 128), 106 and 128
// without that; it costs the largest products nothing and gains them nothing, which the chip's
// power holds.  For the 32 x 128 tile D = 4 where a CU has one workgroup, which would wait for
// memory each stage, and D = 3 where there are more: two then fit its LDS, and one works while
// the other starts or ends (64 rows over 256 experts x 4096 x 2048: 80 us, D = 4 83, D = 2 87;
// 128 rows over 32 experts x 4096 x 7168: 146, 148, 179).

struct TileAt {
    int g;                                        // expert
    int64_t row0;                                 // first row
    int rows;
    int64_t n0;                                   // first feature (of a part)
    int cols;
    uint32_t ntile;
};

// find_tile, but with the tiles in another order: all whole ones, then the experts' last
// partial ones with more than half the rows, then the others.  A workgroup of a kernel whose
// small tiles take less time then comes last.
template <int TM>
__device__ __forceinline__ bool find_tile_whole_first(const int32_t* __restrict__ offs, int G, uint32_t mtile, int& g,
                                                      int64_t& row0, int& rows)
{
    const int lane = threadIdx.x & 63;
    uint32_t run = 0;
    for (int pass = 0; pass < 3; ++pass)
        for (int g0 = 0; g0 < G; g0 += 64) {
            const int h = g0 + lane;
            const int32_t from = offs[min(h, G)], m = offs[min(h + 1, G)] - from;
            const uint32_t whole = (uint32_t)m / TM, rest = (uint32_t)m % TM;
            const uint32_t own = pass == 0 ? whole : (pass == 1) == (rest > TM / 2) && rest ? 1 : 0;
            const uint32_t incl = wave_scan(own), first = run + incl - own;
            const uint64_t mask = __ballot(mtile >= first && mtile - first < own);
            if (mask) {
                const int src = __builtin_ctzll(mask);
                const uint32_t skip = pass == 0 ? mtile - first : whole;
                g = g0 + src;
                row0 = (int64_t)__builtin_amdgcn_readlane(from, src) +
                       (int64_t)TM * (uint32_t)__builtin_amdgcn_readlane((int)skip, src);
                rows = pass == 0 ? TM : __builtin_amdgcn_readlane((int)rest, src);
                return true;
            }
            run += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
        }
    return false;
}

// The workgroup's tile of TM rows and TN rows of the weights; false if it has none.
template <int TM, int TN, int kParts, bool kWholeFirst>
__device__ __forceinline__ bool tile_place(const int32_t* __restrict__ offs, int G, int64_t N, uint32_t ntn, TileAt& at,
                                           bool by_feature = false)
{
    uint32_t mtile;
    // Workgroups go round-robin over the 8 XCDs, so with pairs of token tiles an XCD has every
    // second token tile and every fourth feature tile of a stretch: 8 x 4 of 256 workgroups,
    // all of them on one expert or a few neighbours, and an expert with few rows spread over
    // all XCDs.  (Groups of 4 dealt to one XCD each, as the other GEMM has them: 2048 rows over
    // 32 experts 225 us, here 213; 65536 rows x 7168 x 2048 975, 955; 32768 rows 905, 892.)
    // by_feature: a run of feature tiles to each XCD, with the token tiles inside: weights that
    // are most of the bytes are then read by one XCD.
    if (by_feature) {
        const uint32_t lin = xcd_remap(blockIdx.x, gridDim.x), ntm = gridDim.x / ntn;
        at.ntile = lin / ntm;
        mtile = lin % ntm;
    } else {
        tile_of<2>(blockIdx.x, gridDim.x, ntn, mtile, at.ntile);
    }
    at.n0 = (int64_t)(TN / kParts) * at.ntile;
    at.cols = (int)min((int64_t)(TN / kParts), N - at.n0);
    bool found;
    if constexpr (kWholeFirst)
        found = find_tile_whole_first<TM>(offs, G, mtile, at.g, at.row0, at.rows);
    else
        found = find_tile<TM>(offs, G, mtile, at.g, at.row0, at.rows);
    return found;
}

// A tile's sums, in t: lane (r, h) = (lane % 16, lane / 16) of wave (wm, wn) = (wave % WM,
// wave / WM) holds in acc[mt][nt] those of token 16 (MT wm + mt) + r and tile features
// 16 (NT wn + nt) + 4 h + (0..3).  The LDS arrays are free again afterwards.  lds2 and lds3 are
// the third and fourth buffer, or the late rows of two; every array has a part for each group,
// whose sums are of its blocks alone.
template <class W, int kParts>
__device__ __forceinline__ void tile_sums(uint8_t* lds0, uint8_t* lds1, uint8_t* lds2, uint8_t* lds3,
                                          const uint8_t* __restrict__ a, const float* __restrict__ sa,
                                          const uint8_t* __restrict__ w, const float* __restrict__ sw, int64_t N,
                                          int64_t K, const TileAt& at, typename W::State& t)
{
    constexpr int WM = W::kWM, WN = W::kWN, MT = W::kMT, NT = W::kNT, D = W::kD, TN = W::TN;
    static_assert(kParts == 1 || (WN % 2 == 0 && W::kWaves % 2 == 0), "a wave loads and multiplies one part");
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) % W::kWaves;
    const uint32_t group = W::kSplit == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 6) / W::kWaves;
    const int g = at.g, rows = at.rows, cols = at.cols;
    const int64_t row0 = at.row0, n0 = at.n0;
    const uint32_t kb_n = (uint32_t)((K + kBK - 1) / kBK);
    const uint32_t nb_n = (uint32_t)((N + 127) / 128);
    const int wm = wave % WM, wn = wave / WM;
    const uint32_t r = (uint32_t)(lane & 15), h = (uint32_t)(lane >> 4);

    // loader: instruction i of wave w fills token rows 8 (kLoadsA w + i) .. + 7 (and feature
    // rows alike), or with two halves the same of the early rows and of the late ones, each wave
    // row's MT groups of 8; lane L takes row L / 8 of them and LDS chunk L % 8, the row's chunk
    // (L % 8) ^ ((row >> 1) & 7), which is the same for every other i.  Token scales: slot
    // 64 w + L, which is token tile slot % MT of row slot / MT % 16 of wave row slot / (16 MT)
    const uint32_t l8 = (uint32_t)(lane >> 3), l16 = (uint32_t)(lane >> 4), lc = (uint32_t)(lane & 7);
    const uint32_t al = (uint32_t)(W::kLoadsA * wave) / (W::kHalves ? 2 : 1);      // first 8-row groups: in LDS
    const uint32_t ag = W::kHalves ? 2 * MT * (al / MT) + al % MT : al;            // of the tile
    const uint32_t wg = (uint32_t)(W::kLoadsW * wave);
    const uint32_t slot = (uint32_t)tid % (64 * W::kWaves);
    const uint32_t srow = slot / (16 * MT) * (16 * MT) + slot % MT * 16 + slot / MT % 16;
    // the part that the wave loads, and the one that it multiplies
    const uint32_t lpart = 8 * wg / (TN / kParts), part = (uint32_t)(16 * NT * wn) / (TN / kParts);
    const uint32_t nb = min(((uint32_t)n0 + 16 * NT * wn - part * (TN / kParts)) / 128, nb_n - 1);
    TileCtx<D> cx;
    cx.buf[0] = lds0 + group * W::kBuf;
    cx.buf[1] = lds1 + group * W::kBuf;
    if constexpr (D > 2)
        cx.buf[2] = lds2 + group * W::kBuf2;
    if constexpr (D > 3)
        cx.buf[3] = lds3 + group * W::kBuf3;
    cx.late[0] = lds2 + group * W::kBuf2;         // (of two buffers)
    cx.late[1] = lds3 + group * W::kBuf3;
    cx.ra = strip_rsrc(a + row0 * K, (uint64_t)rows * (uint64_t)K);
    cx.rw = strip_rsrc(w + ((kParts * (int64_t)g + lpart) * N + n0) * K, (uint64_t)cols * (uint64_t)K);
    cx.rsa = strip_rsrc(sa + row0 * kb_n, (uint64_t)rows * kb_n * 4);
    cx.rsw = strip_rsrc(sw + ((kParts * (int64_t)g + part) * nb_n + nb) * kb_n, (uint64_t)kb_n * 4);
    cx.K = (uint32_t)K;
    cx.blocks = kb_n;
    // (every group runs the same number of stages, as they meet at the same barriers)
    const uint32_t stages = (kb_n + W::kSplit - 1) / W::kSplit;
    cx.first = group * stages;
    cx.count = cx.first >= kb_n ? 0 : min(stages, kb_n - cx.first);
    const uint32_t run = W::kSplit == 1 ? kb_n : max(cx.count, 1u);
    cx.turn = K % 4096 == 0 ? (at.ntile + 5 * (uint32_t)g) % run : 0;
    cx.abase = (8 * ag + l8) * cx.K;
    cx.wbase = (8 * wg - lpart * (TN / kParts) + l8) * cx.K;
    cx.ac0 = 16 * (lc ^ ((4 * ag + l16) & 7));
    cx.ac1 = 16 * (lc ^ ((4 * ag + 4 + l16) & 7));
    cx.wc0 = 16 * (lc ^ ((4 * wg + l16) & 7));
    cx.wc1 = 16 * (lc ^ ((4 * wg + 4 + l16) & 7));
    cx.lds_a = 8 * al * kBK;
    cx.lds_w = (W::kTok + 8 * wg) * kBK;
    cx.lds_s = 256 * (uint32_t)wave;
    cx.srow = srow * kb_n * 4;
    cx.sslot = slot;
    cx.arow = (uint32_t)((W::kHalves ? 8 : 16) * MT * wm + r) * kBK;
    cx.wrow = (uint32_t)(W::kTok + 16 * NT * wn + r) * kBK;
    cx.c0 = 16 * (h ^ ((r >> 1) & 7));
    cx.c1 = 16 * ((4 + h) ^ ((r >> 1) & 7));
    cx.scl_at = (16 * (uint32_t)wm + r) * MT;

#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        t.sc[mt] = 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            t.acc[mt][nt] = f32x4{};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        t.p[i] = f32x4{};
#pragma unroll
    for (int b = 0; b < D; ++b) {
        W::issue_scales(cx, b, b);
        W::issue_operands(cx, b, b, 0, W::kLoadsA + W::kLoadsW);
        __builtin_amdgcn_sched_barrier(0);        // (the waits count the loads in this order)
    }
    // (only loads into LDS are counted: those into registers do not return in one order with
    // them; measured: counting over both let a stage start early)
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most((D - 1) * W::kLoads));
    meet();
    W::read_scales(cx, t, 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        t.fw[nt] = W::weight_frag(cx, 0, nt);
    t.fa[0] = W::token_frag(cx, 0, 0);
    // D stages at a time, then the rest one by one (leaving the loop between its stages made
    // the compiler copy the accumulators; running whole turns over zeros took 16.3 us where
    // this takes 15.5, 1501 rows x 1352 x 1744); the loads and reads for a stage past the last
    // find zeros
    uint32_t s = 0;
    for (; s + D <= stages; s += D) {
        W::template stage<0>(cx, t, s);
        W::template stage<1>(cx, t, s + 1);
        if constexpr (D > 2)
            W::template stage<2>(cx, t, s + 2);
        if constexpr (D > 3)
            W::template stage<3>(cx, t, s + 3);
    }
    if (s < stages)
        W::template stage<0>(cx, t, s);
    if constexpr (D > 2)
        if (s + 1 < stages)
            W::template stage<1>(cx, t, s + 1);
    if constexpr (D > 3)
        if (s + 2 < stages)
            W::template stage<2>(cx, t, s + 2);
    W::template add<-3>(t);
    W::template add<-2>(t);
    W::template add<-1>(t);
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0));  // no load into LDS is left
    __syncthreads();
}

// The loop for few rows and few tiles, where a tile's walk along K would be the time: a
// workgroup owns 16 MT tokens x 32 rows of the weights (16 features of each part) and its 4
// waves share K, each a run of blocks that it loads for itself, kAhead blocks ahead, through a
// ring of its own in LDS: no wave waits for another before the end.  The waves' sums meet in
// LDS and are added in wave order.
// What bounds it is what a CU can load (one expert's 16 rows x 2112 x 7168: 8.5 us; straight
// into the fragments' registers, 64 bytes of a row at a time, the same took 14.4).
constexpr int kRowsTN = 32, kRowsWaves = 4;

template <int MT>
struct RowsTile {
    static constexpr int TM = 16 * MT, TN = kRowsTN, NT = TN / 16, kAhead = 4;
    static constexpr int kRow = TN + 4;           // floats of a token's row in LDS
    static constexpr int kStage = (TM + TN) * kBK, kBuf = kStage + 512;   // operands; token scales, the weights'
    static constexpr int kLoads = (TM + TN) / 8 + 2;                      // of a block
    typedef float Part[TM][kRow];

    // The sum of tile features n .. n + 3 of token m.
    static __device__ __forceinline__ f32x4 sum(const Part* part, int m, int n)
    {
        f32x4 v = *reinterpret_cast<const f32x4*>(&part[0][m][n]);
#pragma unroll
        for (int q = 1; q < kRowsWaves; ++q)
            v += *reinterpret_cast<const f32x4*>(&part[q][m][n]);
        return v;
    }
};

// The workgroup's tile of TM rows and kRowsTN rows of the weights; false if it has none.  Feature
// tile by feature tile, token tiles inside: the token tiles of an expert follow each other on
// one XCD and share the weights in its L2.
template <int TM, int kParts>
__device__ __forceinline__ bool rows_place(const int32_t* __restrict__ offs, int G, int64_t N, uint32_t ntm, TileAt& at)
{
    const uint32_t lin = xcd_remap(blockIdx.x, gridDim.x);
    at.ntile = lin / ntm;
    at.n0 = (int64_t)(kRowsTN / kParts) * at.ntile;
    at.cols = (int)min((int64_t)(kRowsTN / kParts), N - at.n0);
    return find_tile<TM>(offs, G, lin % ntm, at.g, at.row0, at.rows);
}

// The waves' sums, in part.
template <int MT, int kParts>
__device__ __forceinline__ void rows_sums(uint8_t* lds0, uint8_t* lds1, uint8_t* lds2, uint8_t* lds3,
                                          typename RowsTile<MT>::Part* part, const uint8_t* __restrict__ a,
                                          const float* __restrict__ sa, const uint8_t* __restrict__ w,
                                          const float* __restrict__ sw, int64_t N, int64_t K, const TileAt& at)
{
    typedef RowsTile<MT> R;
    constexpr int TM = R::TM, TN = R::TN, W = kRowsWaves, NT = R::NT, kAhead = R::kAhead;
    constexpr int kStage = R::kStage, kBuf = R::kBuf, kLoads = R::kLoads;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = at.g, rows = at.rows, cols = at.cols;
    const int64_t row0 = at.row0, n0 = at.n0;
    const uint32_t kb_n = (uint32_t)((K + kBK - 1) / kBK);
    const uint32_t nb_n = (uint32_t)((N + 127) / 128);
    const uint32_t kb0 = kb_n * wave / W, kb1 = kb_n * (wave + 1) / W;
    const uint32_t r = (uint32_t)(lane & 15), h = (uint32_t)(lane >> 4);

    const __amdgpu_buffer_rsrc_t ra = strip_rsrc(a + row0 * K, (uint64_t)rows * (uint64_t)K);
    const uint8_t* const w0 = w + (kParts * (int64_t)g * N + n0) * K;
    const __amdgpu_buffer_rsrc_t rw = strip_rsrc(w0, (uint64_t)cols * (uint64_t)K);
    const __amdgpu_buffer_rsrc_t rw1 = strip_rsrc(w0 + (kParts - 1) * N * K, (uint64_t)cols * (uint64_t)K);
    const __amdgpu_buffer_rsrc_t rsa = strip_rsrc(sa + row0 * kb_n, (uint64_t)rows * kb_n * 4);
    // (the weights' scales of both parts are one array, and every other lane loads the second's)
    const uint64_t next = kParts == 1 ? 0 : (uint64_t)nb_n * kb_n * 4;
    const __amdgpu_buffer_rsrc_t rsw = strip_rsrc(sw + (kParts * (int64_t)g * nb_n + n0 / 128) * kb_n,
                                                  (uint64_t)kb_n * 4 + next);
    const uint32_t my_next = lane & 1 ? (uint32_t)next : 0;

    // as in the tile kernel: a load fills 8 rows, lane L row L / 8 and LDS chunk L % 8 of them
    const uint32_t lrow = (uint32_t)(lane >> 3), lc = (uint32_t)(lane & 7);
    const uint32_t even = 16 * (lc ^ h), odd = 16 * (lc ^ (4 + h));       // chunks of load 0, 2, .. and 1, 3, ..
    const uint32_t c0 = 16 * (h ^ ((r >> 1) & 7)), c1 = 16 * ((4 + h) ^ ((r >> 1) & 7));
    auto load = [&](uint8_t* to, uint32_t kb) {
        // (a block of another wave's run, or past the last, reads nothing)
        const uint32_t k0 = kb < kb1 ? kb * kBK : kOutOfRange;
        const uint32_t oe = even + k0 < (uint32_t)K ? lrow * (uint32_t)K + even : kOutOfRange;
        const uint32_t oo = odd + k0 < (uint32_t)K ? lrow * (uint32_t)K + odd : kOutOfRange;
        const uint32_t kc = kb < kb1 ? k0 : 0;
#pragma unroll
        for (int i = 0; i < (TM + TN) / 8; ++i) {
            const bool tok = i < TM / 8;
            const int in = tok ? i : (i - TM / 8) % (TN / 8 / kParts);
            const bool second = !tok && i - TM / 8 != in;
            load16_to_lds(tok ? ra : second ? rw1 : rw, to + 8 * i * kBK, (i & 1 ? oo : oe) + 8 * in * (uint32_t)K, kc);
        }
        const uint32_t slot = (uint32_t)lane;     // (slots past TM are not read)
        load4_to_lds(rsa, to + kStage, kb < kb1 ? (slot * kb_n + kb) * 4 : kOutOfRange);
        load4_to_lds(rsw, to + kStage + 256, kb < kb1 ? 4 * kb + my_next : kOutOfRange);
    };
    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            acc[mt][nt] = f32x4{};
    uint8_t* const buf[kAhead] = {lds0 + wave * kBuf, lds1 + wave * kBuf, lds2 + wave * kBuf, lds3 + wave * kBuf};
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        load(buf[u], kb0 + u);
    for (uint32_t kb = kb0; kb < kb1; kb += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(vmcnt_at_most((kAhead - 1) * kLoads));
            asm volatile("" ::: "memory");
            i32x8 fw[NT], fa[MT];
            float sc[kParts][MT];
            const float* const scales = reinterpret_cast<const float*>(buf[u] + kStage);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                fw[nt] = frag(buf[u] + (TM + 16 * nt + r) * kBK, c0, c1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                fa[mt] = frag(buf[u] + (16 * mt + r) * kBK, c0, c1);
#pragma unroll
                for (int q = 0; q < kParts; ++q)
                    sc[q][mt] = scales[16 * mt + r] * scales[64 + q];
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");             // all of it is in registers
            load(buf[u], kb + kAhead + u);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const f32x4 p = mfma128(fw[nt], fa[mt], f32x4{});
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[mt][nt][i] = __builtin_fmaf(sc[nt * kParts / NT][mt], p[i], acc[mt][nt][i]);
                }
        }
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0));  // no load into LDS is left
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            *reinterpret_cast<f32x4*>(&part[wave][16 * mt + r][16 * nt + 4 * h]) = acc[mt][nt];
    __syncthreads();
}

}  // namespace mxfp4
