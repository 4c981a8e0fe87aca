// block_gemm.hip -- expert-grouped FP8 product with FP32 block scales.
//
// For the expert g that owns row m (offs[g] <= m < offs[g+1]):
//     y[m, n] = bf16( sum_b sa[m, b] sw_g[n / 128, b] sum_{k in block b} A[m, k] W_g[n, k] )
// A [M, K], W_g [N, K] E4M3, b = k / 128; the last block of K and of N may be partial.
// The matrix cores cannot apply an FP32 scale, so a block's sum has to leave them before it
// is added: v_mfma_f32_16x16x128_f8f6f4 sums a whole block in one instruction from zero, and
// its 4 results per lane go into the FP32 accumulators with one multiply-add each.  With the
// weights as the first operand and the tokens as the second, a lane's results belong to one
// token, so the scale sa sw is one number per lane and token tile.  (Two chained
// v_mfma_f32_32x32x64 per block, 16 results each, measured 1490 us where this form, in the
// first version of the same tile, took 1225.)
//
// What bounds it (32768 rows x 7168 x 4096, 8 experts, 890-950 us, 2.0-2.15 PFLOP/s; this
// library's UE8M0-scaled product of that size, where the matrix cores apply the scales,
// takes 802, the vendor library's per-tensor-scaled FP8 product 710): first the load path (the
// loads alone take 820 us, 590 with every operand in the L2; the products alone 685), then
// power, at 1.92-2.07 GHz with the matrix cores busy half the time (784 us with zeros for
// operands and the clock at its top).  Of a 256 x 256 tile's stage the matrix instructions
// fill 2048 cycles, the scaled adds half as many vector cycles beside them, and its 64 KB have
// to arrive.  With few rows it is the weights' bytes: 128 rows over 32 experts x 4096 x 7168
// take 147-152 us, 6.2-6.4 TB/s.
//
// Two kernels, both with the operands staged in LDS: in the tile kernel all waves share a
// stage, in the rows kernel the waves split K, where there are so few tiles that a tile's walk
// along K would be the time.  Buffer loads take the bounds: rows past the expert's and
// features past N are outside the ranges and read as zero, and a lane whose bytes are past K
// gets an offset outside every range.
#include "block_tile.h"

namespace mxfp4 {

// Half a tile's rows go out through each of two buffers' LDS, kOutRows of them through the
// buffer and the others through its late rows.
template <int WM, int WN, int MT, int NT, int D>
__global__ __launch_bounds__(64 * WM * WN, D == 2 ? 2 : 1) void block_gemm_tile_kernel(
    const uint8_t* __restrict__ a, const float* __restrict__ sa, const uint8_t* __restrict__ w,
    const float* __restrict__ sw, uint16_t* __restrict__ y, const int32_t* __restrict__ offs, int G, int64_t N,
    int64_t K, uint32_t ntn)
{
    typedef Tile<WM, WN, MT, NT, D> W;
    constexpr int TM = W::TM, TN = W::TN, kWaves = W::kWaves;
    constexpr int kOutRows = W::kHalves ? 3 * TM / 8 : TM / 2;
    static_assert(W::kBuf >= kOutRows * TN * 2 && (!W::kHalves || W::kLate >= (TM / 2 - kOutRows) * TN * 2), "out");
    // separate arrays: what is loaded into one does not hold up reads of another
    __shared__ __attribute__((aligned(16))) uint8_t lds0[W::kBuf];
    __shared__ __attribute__((aligned(16))) uint8_t lds1[W::kBuf];
    __shared__ __attribute__((aligned(16))) uint8_t lds2[W::kBuf2];
    __shared__ __attribute__((aligned(16))) uint8_t lds3[W::kBuf3];
    TileAt at;
    if (!tile_place<TM, TN, 1, false>(offs, G, N, ntn, at))
        return;                                   // uniform over the workgroup
    typename W::State t;
    tile_sums<W, 1>(lds0, lds1, lds2, lds3, a, sa, w, sw, N, K, at, t);
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const uint32_t r = (uint32_t)(tid & 15), h = (uint32_t)(tid >> 4 & 3);

    // out through LDS: lane (r, h) of tile (mt, nt) holds token 16 (MT wm + mt) + r and
    // features 16 (NT wn + nt) + 4 h + (0..3); a token's row is 2 TN bytes there with 16-byte
    // chunk c at chunk c ^ (token % 16), then whole row segments go out, 16 bytes a lane
    auto place = [&](uint32_t row) {
        const uint32_t in = row % (TM / 2);
        if (in < (uint32_t)kOutRows)
            return (row < TM / 2 ? lds0 : lds1) + in * (2 * TN);
        return (row < TM / 2 ? lds2 : lds3) + (in - kOutRows) * (2 * TN);
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const f32x4& v = t.acc[mt][nt];
            const bf16x2 p0 = {(__bf16)v[0], (__bf16)v[1]};
            const bf16x2 p1 = {(__bf16)v[2], (__bf16)v[3]};
            const uint32_t c = (uint32_t)(2 * (NT * wn + nt)) + (h >> 1);
            const uint32_t row = (uint32_t)(16 * (MT * wm + mt)) + r;
            *reinterpret_cast<u32x2*>(place(row) + 16 * (c ^ r) + 8 * (h & 1)) =
                u32x2{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1)};
        }
    __syncthreads();
    const __amdgpu_buffer_rsrc_t ry = strip_rsrc(y + at.row0 * N, (uint64_t)at.rows * (uint64_t)N * 2);
    constexpr int kChunks = TN / 8;               // 16-byte chunks of a row
    constexpr int kRows = 64 * kWaves / kChunks;  // rows per pass
    const uint32_t c = (uint32_t)tid % kChunks;
#pragma unroll
    for (int i = 0; i < TM / kRows; ++i) {
        const uint32_t row = (uint32_t)tid / kChunks + kRows * i;
        const uint8_t* const from = place(row) + 16 * (c ^ (row & 15));
        const uint32_t off = (int)(8 * c) < at.cols ? (row * (uint32_t)N + (uint32_t)at.n0) * 2 + 16 * c : kOutOfRange;
        __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4*>(from), ry, (int)off, 0, 2);
    }
}

template <int MT>
__global__ __launch_bounds__(64 * kRowsWaves) void block_gemm_rows_kernel(
    const uint8_t* __restrict__ a, const float* __restrict__ sa, const uint8_t* __restrict__ w,
    const float* __restrict__ sw, uint16_t* __restrict__ y, const int32_t* __restrict__ offs, int G, int64_t N,
    int64_t K, uint32_t ntm)
{
    typedef RowsTile<MT> R;
    // separate arrays: what is loaded into one does not hold up reads of another
    __shared__ __attribute__((aligned(16))) uint8_t lds0[kRowsWaves * R::kBuf];
    __shared__ __attribute__((aligned(16))) uint8_t lds1[kRowsWaves * R::kBuf];
    __shared__ __attribute__((aligned(16))) uint8_t lds2[kRowsWaves * R::kBuf];
    __shared__ __attribute__((aligned(16))) uint8_t lds3[kRowsWaves * R::kBuf];
    __shared__ __attribute__((aligned(16))) typename R::Part part[kRowsWaves];
    TileAt at;
    if (!rows_place<R::TM, 1>(offs, G, N, ntm, at))
        return;                                   // uniform over the workgroup
    rows_sums<MT, 1>(lds0, lds1, lds2, lds3, part, a, sa, w, sw, N, K, at);
    for (int i = threadIdx.x; i < R::TM * R::TN / 4; i += 64 * kRowsWaves) {
        const int m = i / (R::TN / 4), n = i % (R::TN / 4) * 4;
        const f32x4 v = R::sum(part, m, n);
        const bf16x2 p0 = {(__bf16)v[0], (__bf16)v[1]};
        const bf16x2 p1 = {(__bf16)v[2], (__bf16)v[3]};
        if (m < at.rows && n < at.cols)
            *reinterpret_cast<u32x2*>(y + (at.row0 + m) * N + at.n0 + n) =
                u32x2{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1)};
    }
}

hipError_t launch_block_gemm(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, uint16_t* y,
                             const int32_t* offs, int32_t G, int64_t M_cap, int64_t N, int64_t K, hipStream_t stream)
{
    int g = G;
    int64_t n = N, k = K;
    uint32_t nt = 0;                              // feature tiles (tile kernel), token tiles (rows kernel)
    void* args[] = {(void*)&a, (void*)&sa, (void*)&w, (void*)&sw, (void*)&y, (void*)&offs, (void*)&g,
                    (void*)&n, (void*)&k, (void*)&nt};
    auto launch = [&](const void* kernel, int64_t grid, int threads) {
        return grid > 0x7FFFFFFF ? hipErrorInvalidValue
                                 : launch_kernel(kernel, dim3((unsigned)grid), dim3((unsigned)threads), args, stream);
    };
    auto tile = [&](const void* kernel, int TM, int TN, int threads) {
        nt = (uint32_t)((N + TN - 1) / TN);
        return launch(kernel, tiles(M_cap, G, N, TM, TN), threads);
    };
    // The choice goes by the number of workgroups (256 CUs) and the rows an expert has on
    // average, as far as the host knows them: by M_cap.  (Where the rows are far fewer, as on a
    // rank that passes T k for its share, a larger tile than fits is the price: 1033 rows over 32
    // experts x 4096 x 7168 with M_cap 8192 215 us, with M_cap 1033 173; 502 with 4096 168, 161.)
    // Measured in us, the chosen one first:
    //   rows kernel, where each of its workgroups has a CU, or nearly, with 16 tokens or 32: one
    //     expert's 16 rows x 4096 x 7168: 8.8 with 16, 9.5 with 32, 32 x 128 18.8; 32 rows: 9.1,
    //     11.0, 19.0; 64 rows: 11.2 with 32, 15.6 with 16, 32 x 128 19.3; 1 row x 7168 x 2048:
    //     5.8, 7.8; 64 rows over 16 experts x 512 x 4096: 8.7, 12.5; and up to two workgroups of
    //     16 tokens per CU if K is long: 8 rows x 16384 x 7168 25.9, 30.2, but 8 rows x 16384 x
    //     4096 14.8 against 13.0
    //   256 x 256, from 192 rows per expert on: 8 experts, 2048 rows x 4096 x 7168: 102, 128 x
    //     128: 119; 32768 rows: 930, 1160; but 1 expert, 1024 rows x 4096 x 4096 (64 tiles): 49
    //     against 27
    //   128 x 128, from 12 rows on: 8 experts, 256 rows x 7168 x 2048: 27, 32 x 128 32; 3
    //     experts, 1501 rows x 1352 x 1744: 14.9, 20.5; 32 experts, 512 rows x 4096 x 7168: 171,
    //     175
    //   32 x 128 for the rest (32 experts, 128 rows: 146, 128 x 128 158; 1 expert, 200 rows x
    //     4096 x 7168: 20.3, 33), four buffers while there is one workgroup per CU (5 experts'
    //     rows x 4096 x 7168: 30.7, three buffers 35.1)
    const int64_t rows16 = tiles(M_cap, G, N, 16, kRowsTN), rows32 = tiles(M_cap, G, N, 32, kRowsTN);
    if (rows16 <= 320 || (rows16 <= 512 && rows32 > 320 && K > 4096)) {
        nt = (uint32_t)tiles(M_cap, G, 1, 16, 1);
        return launch((const void*)block_gemm_rows_kernel<1>, rows16, 64 * kRowsWaves);
    }
    if (rows32 <= 320) {
        nt = (uint32_t)tiles(M_cap, G, 1, 32, 1);
        return launch((const void*)block_gemm_rows_kernel<2>, rows32, 64 * kRowsWaves);
    }
    if (M_cap >= 192 * (int64_t)G && tiles(M_cap, G, N, 256, 256) >= 192)
        return tile((const void*)block_gemm_tile_kernel<2, 4, 8, 4, 2>, 256, 256, 512);
    if (M_cap >= 12 * (int64_t)G && tiles(M_cap, G, N, 128, 128) >= 128)
        return tile((const void*)block_gemm_tile_kernel<2, 2, 4, 4, 2>, 128, 128, 256);
    if (tiles(M_cap, G, N, 32, 128) <= 256)
        return tile((const void*)block_gemm_tile_kernel<1, 4, 2, 2, 4>, 32, 128, 256);
    return tile((const void*)block_gemm_tile_kernel<1, 4, 2, 2, 3>, 32, 128, 256);
}

}  // namespace mxfp4
