// act_rows.hip -- the gradient of act(p) with p = rows + bias_g, for rows in expert order:
//     dp = dout act'(p),   dbias_g = the sum of dp over the rows of expert g
// dp leaves as BF16, or as E4M3 rows with an FP32 scale per 1x128 block (both from the FP32
// value; the bias takes that one too).
//
// What bounds it is its bytes: 32768 rows of 8 experts x 4096, BF16 out and the bias, 97 us
// without an activation (537 MB, 5.5 TB/s), 145 with GELU (805 MB, 5.6 TB/s).  A thread has eight
// columns and every eighth row of a tile, 32 threads a row's 512 bytes, so that the columns' sums
// stay in registers until the tile's end, where the eight rows of threads meet in LDS.  A tile is
// 32 rows of one expert, which a thread loads all at once, and its sums go to the workspace, where
// a second launch adds them, tile by tile in a fixed order (no atomics: the same call gives the
// same bits); with few rows a workgroup takes all rows of an expert and writes the sums itself.
// (Rows of a tile, 32768 rows of 8 experts x 7168, GELU: 16 351 us, 32 253, 64 260, 128 272; 8192
// x 2048: 34, 24, 24, 30.  32 is best at every size tried above 12 us, of 4 widths and 4
// activations; below, where the launches are the time, they differ by what two timings do.)
#include "activation.h"
#include "tiles.h"

namespace mxfp4 {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kTileRows = 32;
constexpr int kActCols = 256, kLanes = kActCols / 8, kRowGroups = kThreads / kLanes;
constexpr int kBatch = 4;                         // rows of a thread in flight
constexpr int kSumCols = 64, kSumSplit = 16;      // second launch: columns and tile runs of a workgroup
constexpr uint32_t kNowhere = 0x80000000u;        // offset past every buffer's range

}  // namespace

// ALL: a workgroup has all rows of an expert, not a tile of them.
template <bool ALL>
__global__ __launch_bounds__(kThreads) void act_rows_kernel(
    const uint16_t* dout, const uint16_t* pre, uint16_t* dpre, uint8_t* q, float* q_scales, float* sums,
    const int32_t* __restrict__ offs, int G, uint32_t N, uint32_t strips, int act)
{
    __shared__ __attribute__((aligned(16))) float part[kRowGroups][kActCols];
    const uint32_t tile = blockIdx.x / strips, n0 = blockIdx.x % strips * kActCols;
    int g;
    int64_t row0;
    int rows;
    if constexpr (ALL) {
        g = (int)tile;
        row0 = offs[g];
        rows = offs[g + 1] - (int)row0;
    } else if (!find_tile<kTileRows>(offs, G, tile, g, row0, rows)) {
        return;                                   // uniform over the workgroup
    }
    const uint32_t tid = threadIdx.x, c = tid % kLanes, group = tid / kLanes, col = n0 + 8 * c;
    const uint64_t bytes = (uint64_t)rows * N * 2;
    const uint32_t blocks = (N + 127) / 128;
    const __amdgpu_buffer_rsrc_t rd = strip_rsrc(dout + row0 * N, bytes);
    const __amdgpu_buffer_rsrc_t rp = strip_rsrc(pre ? pre + row0 * N : nullptr, pre ? bytes : 0);
    const __amdgpu_buffer_rsrc_t ro = strip_rsrc(dpre ? dpre + row0 * N : nullptr, dpre ? bytes : 0);
    const __amdgpu_buffer_rsrc_t rq = strip_rsrc(q ? q + row0 * N : nullptr, q ? bytes / 2 : 0);
    const __amdgpu_buffer_rsrc_t rs = strip_rsrc(q ? q_scales + row0 * blocks : nullptr,
                                                 q ? (uint64_t)rows * blocks * 4 : 0);
    const bool there = col < N;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int first = 0; first < rows; first += kBatch * kRowGroups) {
        u32x4 d[kBatch], p[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t row = (uint32_t)first + group + kRowGroups * i;
            const int off = there ? (int)((row * N + col) * 2) : (int)kNowhere;
            d[i] = __builtin_amdgcn_raw_buffer_load_b128(rd, off, 0, 2);
            p[i] = act != kActNone ? __builtin_amdgcn_raw_buffer_load_b128(rp, off, 0, 2) : u32x4{};
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t row = (uint32_t)first + group + kRowGroups * i;
            float v[8], x[8], slope[8];
            from_bf16(d[i], v);
            from_bf16(p[i], x);
            activate8<true>(act, x, slope);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] *= slope[j];
                sum[j] += v[j];
            }
            // (rows past the last are outside the ranges: they read zeros and store nothing)
            const uint32_t at = row * N + col;
            if (dpre)
                __builtin_amdgcn_raw_buffer_store_b128(to_bf16(v), ro, there ? (int)(2 * at) : (int)kNowhere, 0, 2);
            if (q) {
                float scale;
                const u32x2 b = to_fp8(v, scale);
                __builtin_amdgcn_raw_buffer_store_b64(b, rq, there ? (int)at : (int)kNowhere, 0, 2);
                __builtin_amdgcn_raw_buffer_store_b32(
                    __float_as_uint(scale), rs,
                    there && col % 128 == 0 ? (int)((row * blocks + col / 128) * 4) : (int)kNowhere, 0, 0);
            }
        }
    }
    if (!sums)
        return;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        *reinterpret_cast<f32x4*>(&part[group][8 * c + 4 * j]) = f32x4{sum[4 * j], sum[4 * j + 1], sum[4 * j + 2],
                                                                       sum[4 * j + 3]};
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kRowGroups; ++i)
        s += part[i][tid];
    if (n0 + tid < N)
        sums[(uint64_t)tile * N + n0 + tid] = s;
}

// dbias_g = the sum of its tiles' sums.
__global__ __launch_bounds__(kSumCols* kSumSplit) void bias_sum_kernel(
    const float* __restrict__ sums, float* __restrict__ dbias, const int32_t* __restrict__ offs, uint32_t N,
    uint32_t strips)
{
    __shared__ float part[kSumSplit][kSumCols];
    const int g = (int)(blockIdx.x / strips);
    const int lane = threadIdx.x & 63;
    const uint32_t run = threadIdx.x / kSumCols, col = blockIdx.x % strips * kSumCols + threadIdx.x % kSumCols;
    uint64_t first = 0;                           // tiles of the experts before
    for (int e0 = 0; e0 < g; e0 += 64) {
        const int e = e0 + lane;
        const uint32_t n = e < g ? ((uint32_t)(offs[e + 1] - offs[e]) + kTileRows - 1) / kTileRows : 0;
        first += (uint32_t)__builtin_amdgcn_readlane((int)wave_scan(n), 63);
    }
    const uint32_t n = ((uint32_t)(offs[g + 1] - offs[g]) + kTileRows - 1) / kTileRows;
    const uint32_t t0 = (uint32_t)((uint64_t)n * run / kSumSplit), t1 = (uint32_t)((uint64_t)n * (run + 1) / kSumSplit);
    float s = 0.0f;
    if (col < N) {
        const float* const from = sums + first * N + col;
#pragma unroll 8
        for (uint32_t t = t0; t < t1; ++t)
            s += from[(uint64_t)t * N];
    }
    part[run][threadIdx.x % kSumCols] = s;
    __syncthreads();
    if (threadIdx.x < kSumCols && col < N) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < kSumSplit; ++i)
            s += part[i][threadIdx.x];
        dbias[(uint64_t)g * N + col] = s;
    }
}

// Whether sums go to the workspace and a second launch, or a workgroup takes all rows of an
// expert, which is faster while those are few: 256 rows of 16 experts x 7168, GELU: 8.4 us, in
// tiles 14.2; 512 of 32: 9.5, 21.7; 64 of one: 8.0, 10.7; but 128 of one: 12.5, 10.7, and 384 of 4:
// 15.4, 11.3 (without an activation 8.1, 10.8 and 8.8, 11.0).  The rows may all be one expert's,
// so there is a limit (512 of 4, hardly split, 18.8, 11.5).
bool act_rows_uses_workspace(int32_t G, int64_t M_cap)
{
    return M_cap > 64 * (int64_t)G || M_cap > 512;
}

namespace {

int64_t act_tiles(int32_t G, int64_t M_cap)
{
    const int64_t live = G < M_cap ? G : M_cap;
    return (M_cap + live * (kTileRows - 1)) / kTileRows;
}

}  // namespace

// Bytes that a call with bias gradients and every one of fewer rows use at most.
int64_t act_rows_workspace(int32_t G, int64_t M_cap, int64_t N)
{
    return act_rows_uses_workspace(G, M_cap) ? 4 * act_tiles(G, M_cap) * N : 0;
}

hipError_t launch_act_rows_backward(const uint16_t* dout, const uint16_t* pre, uint16_t* dpre, uint8_t* q,
                                    float* q_scales, float* dbias, float* work, const int32_t* offs, int32_t G,
                                    int64_t M_cap, int64_t N, int act, hipStream_t stream)
{
    const bool all = dbias && !act_rows_uses_workspace(G, M_cap);
    uint32_t n = (uint32_t)N, strips = (uint32_t)((N + kActCols - 1) / kActCols);
    int g = G;
    float* sums = dbias ? all ? dbias : work : nullptr;
    const int64_t grid = (all ? G : act_tiles(G, M_cap)) * (int64_t)strips;
    const int64_t columns = (N + kSumCols - 1) / kSumCols;
    const bool then = dbias && !all;
    if (grid > 0x7FFFFFFF || (then && G * columns > 0x7FFFFFFF))
        return hipErrorInvalidValue;
    void* args[] = {(void*)&dout, (void*)&pre, (void*)&dpre, (void*)&q, (void*)&q_scales, (void*)&sums,
                    (void*)&offs, (void*)&g, (void*)&n, (void*)&strips, (void*)&act};
    if (grid > 0) {
        const void* const kernel = all ? (const void*)act_rows_kernel<true> : (const void*)act_rows_kernel<false>;
        const hipError_t e = launch_kernel(kernel, dim3((unsigned)grid), dim3(kThreads), args, stream, !then);
        if (e != hipSuccess)
            return e;
    }
    if (!then)
        return hipSuccess;
    uint32_t sum_strips = (uint32_t)columns;
    void* more[] = {(void*)&work, (void*)&dbias, (void*)&offs, (void*)&n, (void*)&sum_strips};
    return launch_kernel((const void*)bias_sum_kernel, dim3((unsigned)(G * columns)), dim3(kSumCols * kSumSplit), more,
                         stream);
}

}  // namespace mxfp4
