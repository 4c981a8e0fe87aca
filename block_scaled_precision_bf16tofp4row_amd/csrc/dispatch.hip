// dispatch.hip -- BF16 token rows quantized into expert order, and the same FP8 quantizer
// for rows that are in expert order already.
//
// Formats:
//   MXFP4 (as the row quantizer of this library writes it: technical summary section 2,
//     items 1-2 of "Practical FP4 Training for Large-Scale MoE Models on Hopper GPUs",
//     activations quantized right before they go to their experts): 32-element blocks,
//     shared exponent floor(log2 amax) - 2, E2M1 nearest even, saturating;
//   E4M3 with one FP32 scale per 1x128 block: with a = max(amax, 2^-100),
//     scale = a / 448 and byte = E4M3(x * (448 / a)), nearest even.  The floor keeps both
//     quotients normal FP32 numbers, so a block of zeros needs no case of its own.
//
// The work goes by token: a row is read and quantized once and written to each of its up
// to k places, so the reads are the tokens' bytes and not the routed rows'.  A lane takes 16
// consecutive elements (two 16-byte loads; its FP8 bytes are one 16-byte store, its codes an
// 8-byte one), a row a multiple of 8 lanes, so a block's amax is exchanged over 8 lanes (FP8)
// or 2 (MXFP4) by DPP.  Where a row is a multiple of 64 lanes a wave has one token, whose
// positions are scalar loads; else rows follow each other without a gap (32768 rows of 128
// elements to 8 places: 21.4 us with a wave per row, 10.8 without).  What bounds it is the writing,
// streamed past the caches: 8192 rows of 7168 to 8 places each take 110 us for 602 MB, 125
// with ordinary stores.  In place, 65536 rows x 7168: 233 us for 1424 MB, x 2048: 68 for 407;
// 512 x 2048: 2.8.
#include "common.h"

namespace mxfp4 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kRowHalfMirror = 0x141;             // DPP: lane i of 8 takes lane 7 - i

__device__ __forceinline__ uint32_t mag_max8(u32x4 v)
{
    u16x2 a = __builtin_bit_cast(u16x2, v.x & 0x7FFF7FFFu);
    u16x2 b = __builtin_bit_cast(u16x2, v.y & 0x7FFF7FFFu);
    u16x2 c = __builtin_bit_cast(u16x2, v.z & 0x7FFF7FFFu);
    u16x2 d = __builtin_bit_cast(u16x2, v.w & 0x7FFF7FFFu);
    u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(a, b), __builtin_elementwise_max(c, d));
    return max((uint32_t)m.x, (uint32_t)m.y);
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Four BF16 (two dwords) times `mul` -> four E4M3 bytes.
__device__ __forceinline__ uint32_t fp8_of4(uint32_t a, uint32_t b, float mul)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(a) * mul, bf16_hi(a) * mul, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(b) * mul, bf16_hi(b) * mul, w, true);
}

// The 16 bytes of one lane of a 1x128 block and its scale (lanes 8 q .. 8 q + 7 hold a block;
// elements past the row are zero).
struct Fp8Lane {
    u32x4 bytes;
    float scale;
};
__device__ __forceinline__ Fp8Lane fp8_lane(u32x4 v0, u32x4 v1)
{
    uint32_t m = quad_max_u32(max(mag_max8(v0), mag_max8(v1)));
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, kRowHalfMirror, 0xF, 0xF, false));
    const float a = fmaxf(__uint_as_float(m << 16), 0x1p-100f);
    const float mul = 448.0f / a;
    return {u32x4{fp8_of4(v0.x, v0.y, mul), fp8_of4(v0.z, v0.w, mul), fp8_of4(v1.x, v1.y, mul),
                  fp8_of4(v1.z, v1.w, mul)},
            a / 448.0f};
}

__device__ __forceinline__ bf16x2 as_bf16x2(uint32_t u)
{
    bf16x2 r;
    __builtin_memcpy(&r, &u, sizeof(r));
    return r;
}

// Eight BF16 -> eight E2M1 codes under the UE8M0 byte s (gfx950's scaled convert: nearest
// even, saturating at +-6; only the exponent of its scale operand counts).
__device__ __forceinline__ uint32_t fp4_of8(u32x4 v, int s)
{
    const float scale = __uint_as_float((uint32_t)s << 23);
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, as_bf16x2(v.x), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(v.y), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(v.z), scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(v.w), scale, 3);
}

}  // namespace

// A lane's number (64 lanes of 16 elements to a unit of the flat work) -> its token and place.
struct Place {
    int64_t t;
    uint32_t lane;                                // of the row
};
template <bool kWhole>
__device__ __forceinline__ Place place_of(uint32_t row_lanes)
{
    // rows of whole waves: the wave's number by the waves of a row, on the scalar unit
    const uint32_t per = kWhole ? row_lanes / 64 : row_lanes;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t u = kWhole ? (uint64_t)blockIdx.x * (kThreads / 64) + wave
                              : (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    uint64_t t;
    if (gridDim.x < (1u << 24))                   // 32 bits hold every u
        t = (uint32_t)u / per;
    else
        t = u / per;
    const uint32_t rest = (uint32_t)(u - t * per);
    return {(int64_t)t, kWhole ? rest * 64 + (threadIdx.x & 63) : rest};
}

// kFp4: MXFP4 codes and UE8M0 bytes, else E4M3 bytes and FP32 scales.  kInPlace: row t
// goes to row t for t < offs[G]; else choice j of token t goes to row pos[t k + j] if that
// is a row of the output.  kWhole: row_lanes is a multiple of 64.
template <bool kFp4, bool kInPlace, bool kWhole>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(
    const uint16_t* __restrict__ x, const int32_t* __restrict__ pos, uint8_t* __restrict__ y,
    void* __restrict__ y_scales, const int32_t* __restrict__ offs, int G, int64_t n_tokens, int k, int64_t M_cap,
    int64_t K, uint32_t row_lanes)
{
    const Place at = place_of<kWhole>(row_lanes);
    const int64_t t = at.t;
    const uint32_t lane = at.lane;                // its lowest 3 bits are the hardware lane's
    const int64_t e0 = 16 * (int64_t)lane;
    const bool here = t < n_tokens && (!kInPlace || t < offs[G]);
    const bool in = here && e0 < K;               // K is a multiple of 16
    u32x4 v0 = {0, 0, 0, 0}, v1 = {0, 0, 0, 0};
    if (in) {
        const u32x4* const p = reinterpret_cast<const u32x4*>(x + t * K + e0);
        v0 = load_stream(p);
        v1 = load_stream(p + 1);
    }
    // (lanes past the row's end stay: those of its last block exchange with them)
    if (!kWhole || here) {
        const int n = kInPlace ? 1 : k;
        if (kFp4) {
            uint32_t m = max(mag_max8(v0), mag_max8(v1));
            m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, kQuadSwap1, 0xF, 0xF, false));
            const int s = max((int)(m >> 7) - 2, 0);
            const u32x2 codes = {fp4_of8(v0, s), fp4_of8(v1, s)};
            for (int j = 0; j < n; ++j) {
                const int64_t row = !here ? -1 : kInPlace ? t : (int64_t)pos[t * k + j];
                if (!in || row < 0 || row >= M_cap)
                    continue;
                store_stream(reinterpret_cast<u32x2*>(y + (row * K + e0) / 2), codes);
                if (!(lane & 1))
                    static_cast<uint8_t*>(y_scales)[(row * K + e0) / 32] = (uint8_t)s;
            }
        } else {
            const Fp8Lane q = fp8_lane(v0, v1);
            const int64_t kb = (K + 127) / 128;
            for (int j = 0; j < n; ++j) {
                const int64_t row = !here ? -1 : kInPlace ? t : (int64_t)pos[t * k + j];
                if (!in || row < 0 || row >= M_cap)
                    continue;
                store_stream(reinterpret_cast<u32x4*>(y + row * K + e0), q.bytes);
                if (!(lane & 7))
                    static_cast<float*>(y_scales)[row * kb + e0 / 128] = q.scale;
            }
        }
    }
}

template <bool kFp4, bool kInPlace>
static hipError_t launch_dispatch_kernel(const uint16_t* x, const int32_t* pos, uint8_t* y, void* y_scales,
                                         const int32_t* offs, int32_t G, int64_t T, int32_t k, int64_t M_cap,
                                         int64_t K, hipStream_t stream)
{
    const int64_t lanes = (K + 127) / 128 * 8;
    const int64_t grid = (T * lanes + kThreads - 1) / kThreads;
    if (grid > 0x7FFFFFFF)
        return hipErrorInvalidValue;
    uint32_t row_lanes = (uint32_t)lanes;
    int g = G, kk = k;
    int64_t t = T, cap = M_cap, w = K;
    void* args[] = {(void*)&x, (void*)&pos, (void*)&y, (void*)&y_scales, (void*)&offs, (void*)&g,
                    (void*)&t, (void*)&kk, (void*)&cap, (void*)&w, (void*)&row_lanes};
    const void* kern = lanes % 64 == 0 ? (const void*)dispatch_kernel<kFp4, kInPlace, true>
                                       : (const void*)dispatch_kernel<kFp4, kInPlace, false>;
    return launch_kernel(kern, dim3((unsigned)grid), dim3(kThreads), args, stream);
}

hipError_t launch_dispatch_rows(const uint16_t* x, const int32_t* pos, uint8_t* codes, uint8_t* scales, int64_t T,
                                int32_t k, int64_t M_cap, int64_t K, hipStream_t stream)
{
    return launch_dispatch_kernel<true, false>(x, pos, codes, scales, nullptr, 0, T, k, M_cap, K, stream);
}

hipError_t launch_dispatch_fp8_rows(const uint16_t* x, const int32_t* pos, uint8_t* y, float* y_scales, int64_t T,
                                    int32_t k, int64_t M_cap, int64_t K, hipStream_t stream)
{
    return launch_dispatch_kernel<false, false>(x, pos, y, y_scales, nullptr, 0, T, k, M_cap, K, stream);
}

hipError_t launch_fp8_rows_f32(const uint16_t* x, uint8_t* y, float* y_scales, const int32_t* offs, int32_t G,
                               int64_t M_cap, int64_t K, hipStream_t stream)
{
    return launch_dispatch_kernel<false, true>(x, nullptr, y, y_scales, offs, G, M_cap, 1, M_cap, K, stream);
}

}  // namespace mxfp4
