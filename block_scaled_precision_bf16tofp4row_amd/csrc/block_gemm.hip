// block_gemm.hip -- expert-grouped FP8 product with FP32 block scales.
//
// For the expert g that owns row m (offs[g] <= m < offs[g+1]):
//     y[m, n] = bf16( sum_b sa[m, b] sw_g[n / 128, b] sum_{k in block b} A[m, k] W_g[n, k] )
// A [M, K], W_g [N, K] E4M3, b = k / 128; the last block of K and of N may be partial.
// The matrix cores cannot apply an FP32 scale, so each 128-block of K is summed by two
// v_mfma_f32_32x32x64_f8f6f4 from zero and added to the FP32 accumulators under its scale
// (16 multiply-adds of the vector unit per two 64-cycle matrix instructions).  With the
// weights as the first operand and the tokens as the second, a lane's 16 results belong to
// one token, so the scale sa sw is one number per lane and tile.
//
// A workgroup owns a TM x TN tile of one expert and walks K in stages of 128 through two
// LDS buffers: the next stage's operand bytes go from memory to LDS (buffer_load ... lds)
// while the present one is multiplied.  LDS rows are 128 bytes with 16-byte chunk c of row
// r at chunk c ^ ((r >> 1) & 7), so that the fragment reads of 16 rows hit distinct banks.
// Rows past the expert's and features past N are outside the buffers' ranges and read as
// zero; so are a row's bytes past K (their lanes' offsets are put out of range).
#include "tiles.h"

namespace mxfp4 {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kBK = 128;                          // K per stage: one scale block
constexpr uint32_t kOutOfRange = 0x80000000u;     // offset past every buffer's range
constexpr int kUnitScale = 0x7F7F7F7F;            // E8M0 bytes of 1.0

// A lane's fragment of one operand row for 64 of K: the row's 16-byte LDS chunks at byte
// offsets c0 and c1.
__device__ __forceinline__ i32x8 frag(const uint8_t* rowp, uint32_t c0, uint32_t c1)
{
    const u32x4 v0 = *reinterpret_cast<const u32x4*>(rowp + c0);
    const u32x4 v1 = *reinterpret_cast<const u32x4*>(rowp + c1);
    return i32x8{(int)v0.x, (int)v0.y, (int)v0.z, (int)v0.w, (int)v1.x, (int)v1.y, (int)v1.z, (int)v1.w};
}

__device__ __forceinline__ f32x16 mfma64(i32x8 w, i32x8 a, f32x16 c)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, c, 0, 0, 0, kUnitScale, 0, kUnitScale);
}

}  // namespace

// WM x WN waves; a wave computes MT x NT tiles of 32 tokens x 32 features.
template <int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 1) void block_gemm_kernel(
    const uint8_t* __restrict__ a, const float* __restrict__ sa, const uint8_t* __restrict__ w,
    const float* __restrict__ sw, uint16_t* __restrict__ y, const int32_t* __restrict__ offs, int G, int64_t N,
    int64_t K, uint32_t ntn)
{
    constexpr int MT = TM / WM / 32, NT = TN / WN / 32;
    constexpr int kStage = (TM + TN) * kBK;
    constexpr int kLoads = (TM + TN) / 8 / (WM * WN);       // 8-row loads of a wave per stage
    static_assert(128 % (32 * NT) == 0 && TN % 128 == 0, "a wave's features lie in one scale block");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][kStage];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t mtile, ntile;
    tile_of(group_interleave(blockIdx.x, gridDim.x, kGroupM * ntn), gridDim.x, ntn, mtile, ntile);
    int g;
    int64_t row0;
    int rows;
    if (!find_tile<TM>(offs, G, mtile, g, row0, rows))
        return;                                   // uniform over the workgroup
    const int64_t n0 = (int64_t)TN * ntile;
    const int cols = (int)min((int64_t)TN, N - n0);
    const uint32_t kb_n = (uint32_t)((K + kBK - 1) / kBK);
    const uint32_t nb_n = (uint32_t)((N + 127) / 128);

    const __amdgpu_buffer_rsrc_t ra = strip_rsrc(a + row0 * K, (uint64_t)rows * (uint64_t)K);
    const __amdgpu_buffer_rsrc_t rw = strip_rsrc(w + ((int64_t)g * N + n0) * K, (uint64_t)cols * (uint64_t)K);
    const __amdgpu_buffer_rsrc_t rsa = strip_rsrc(sa + row0 * kb_n, (uint64_t)rows * kb_n * 4);

    // loader: instruction i of wave w fills rows 8 (kLoads w + i) .. + 7 of the stage (tokens,
    // then features); lane L takes row L / 8 of them and LDS chunk L % 8
    uint32_t loff[kLoads], lcol[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const uint32_t lrow = (uint32_t)(8 * (kLoads * wave + i) + (lane >> 3));
        const uint32_t r = lrow < TM ? lrow : lrow - TM;
        lcol[i] = 16 * ((uint32_t)(lane & 7) ^ ((lrow >> 1) & 7));
        loff[i] = r * (uint32_t)K + lcol[i];
    }
    auto issue = [&](uint32_t s, int buf) {
        typedef __attribute__((address_space(3))) uint8_t lds_u8;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int row8 = 8 * (kLoads * wave + i);
            const uint32_t off = lcol[i] + s * kBK < (uint32_t)K ? loff[i] : kOutOfRange;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(row8 < TM ? ra : rw, (lds_u8*)lds[buf] + row8 * kBK, 16, off,
                                                     (int)(s * kBK), 0, 0);
        }
    };

    const int wm = wave % WM, wn = wave / WM;
    const uint32_t r = (uint32_t)(lane & 31), h = (uint32_t)(lane >> 5);
    const uint32_t sw8 = (r >> 1) & 7;            // the swizzle of rows r + 32 x
    // scales: a lane's tokens, and the wave's block of features
    const uint32_t nb = min((uint32_t)(n0 + 32 * NT * wn) / 128, nb_n - 1);
    const float* const swp = sw + ((int64_t)g * nb_n + nb) * kb_n;
    uint32_t soff[MT];
    float sc[MT], sc_next[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        soff[mt] = (uint32_t)(32 * (MT * wm + mt) + r) * kb_n * 4;
    auto load_scales = [&](uint32_t s, float (&to)[MT]) {
        const float b = swp[s];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            to[mt] = b * __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rsa, (int)soff[mt], (int)(4 * s), 0));
    };

    f32x16 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            acc[mt][nt] = f32x16{};

    issue(0, 0);
    load_scales(0, sc);
    for (uint32_t s = 0; s < kb_n; ++s) {
        const int buf = s & 1;
        __builtin_amdgcn_s_waitcnt(0x0F70);       // vmcnt(0): this lane's loads of stage s are in LDS
        __syncthreads();                          // everybody's are, and the other buffer is read
        if (s + 1 < kb_n) {
            issue(s + 1, buf ^ 1);
            load_scales(s + 1, sc_next);
        }
        i32x8 fw[2][NT];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t c0 = 16 * ((4 * j + h) ^ sw8), c1 = 16 * ((4 * j + 2 + h) ^ sw8);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                fw[j][nt] = frag(lds[buf] + (TM + 32 * (NT * wn + nt) + r) * kBK, c0, c1);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            i32x8 fa[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                fa[j] = frag(lds[buf] + (32 * (MT * wm + mt) + r) * kBK, 16 * ((4 * j + h) ^ sw8),
                             16 * ((4 * j + 2 + h) ^ sw8));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                f32x16 p = mfma64(fw[0][nt], fa[0], f32x16{});
                p = mfma64(fw[1][nt], fa[1], p);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[mt][nt][i] = __builtin_fmaf(sc[mt], p[i], acc[mt][nt][i]);
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            sc[mt] = sc_next[mt];
    }

    // lane (r, h) of tile (mt, nt) holds token 32 (MT wm + mt) + r and features
    // 32 (NT wn + nt) + 8 q + 4 h + (0..3) in values 4q .. 4q + 3; N is a multiple of 8
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int m = 32 * (MT * wm + mt) + (int)r;
        if (m >= rows)
            continue;
        uint16_t* const yrow = y + (row0 + m) * N + n0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = 32 * (NT * wn + nt) + 8 * q + 4 * (int)h;
                const f32x16& v = acc[mt][nt];
                const bf16x2 p0 = {(__bf16)v[4 * q + 0], (__bf16)v[4 * q + 1]};
                const bf16x2 p1 = {(__bf16)v[4 * q + 2], (__bf16)v[4 * q + 3]};
                if (n < cols)
                    *reinterpret_cast<u32x2*>(yrow + n) =
                        u32x2{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1)};
            }
    }
}

hipError_t launch_block_gemm(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, uint16_t* y,
                             const int32_t* offs, int32_t G, int64_t M_cap, int64_t N, int64_t K, hipStream_t stream)
{
    constexpr int TM = 64, TN = 128;
    uint32_t ntn = (uint32_t)((N + TN - 1) / TN);
    const int64_t grid = ((M_cap + TM - 1) / TM + G) * ntn;
    if (grid > 0x7FFFFFFF)
        return hipErrorInvalidValue;
    int g = G;
    int64_t n = N, k = K;
    void* args[] = {(void*)&a, (void*)&sa, (void*)&w, (void*)&sw, (void*)&y, (void*)&offs, (void*)&g,
                    (void*)&n, (void*)&k, (void*)&ntn};
    return launch_kernel((const void*)block_gemm_kernel<TM, TN, 1, 4>, dim3((unsigned)grid), dim3(256), args, stream);
}

}  // namespace mxfp4
