// combine.hip -- the experts' rows back to their tokens, and the gradients of that.
//
//     out[t] = base[t] + sum_j w[t, j] Y[pos[t, j]]          (base, w optional; w = 1)
//     dY[pos[t, j]] = w[t, j] dout[t],   dw[t, j] = <dout[t], Y[pos[t, j]]>
// over the choices j with a row (0 <= pos < M_cap); sums in FP32, j ascending, rounded once
// to BF16 (nearest even), so a result does not depend on the launch.  The dispatch's own
// gradient is the first line with w = 1 on the routed rows' gradients.
//
// Both move each routed row once, and its bytes are what bounds them (8192 tokens x 7168, 8
// choices and a base: 199 us, 5.9 TB/s; backward: 380 us, 5.2 TB/s).  A lane takes 8
// elements (16 bytes) of a token; the positions are loaded one per lane and the choices
// without a row dropped by a ballot, so that the loop over the others has its row loads
// (kBatch of them) in flight together.
#include "lanes.h"

namespace mxfp4 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kBatch = 8;                         // routed rows in flight per wave

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const bf16x2 p = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ u32x4 pack8(const float (&v)[8])
{
    return u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
}
__device__ __forceinline__ void unpack8(u32x4 u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}

// Lane j's choice of token t, and the choices that have a row.
struct Choices {
    int32_t row;
    float w;
    uint64_t live;
};
__device__ __forceinline__ Choices choices_of(const int32_t* __restrict__ pos, const float* __restrict__ weights,
                                              int64_t t, int k, int64_t M_cap)
{
    const int lane = threadIdx.x & 63;
    Choices c{-1, 1.0f, 0};
    if (lane < k) {
        c.row = pos[t * k + lane];
        if (weights)
            c.w = weights[t * k + lane];
    }
    c.live = __ballot(c.row >= 0 && c.row < M_cap);
    return c;
}

}  // namespace

__global__ __launch_bounds__(kThreads) void combine_kernel(
    const uint16_t* __restrict__ y, const int32_t* __restrict__ pos, const float* __restrict__ weights,
    const uint16_t* __restrict__ base, uint16_t* __restrict__ out, int64_t n_tokens, int k, int64_t M_cap, int64_t K,
    uint32_t units)
{
    const int lane = threadIdx.x & 63;
    const int64_t u = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = u / units;
    if (t >= n_tokens)
        return;
    const int64_t e0 = (u - t * units) * 512 + 8 * lane;
    const bool in = e0 < K;                       // K is a multiple of 8
    const int64_t el = in ? e0 : 0;               // lanes past the row read its start and write nothing
    const Choices c = choices_of(pos, weights, t, k, M_cap);
    float acc[8] = {};
    if (base)
        unpack8(load_stream(reinterpret_cast<const u32x4*>(base + t * K + el)), acc);
    for (uint64_t left = c.live; left;) {
        u32x4 v[kBatch];
        float w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            w[i] = 0.0f;
            v[i] = u32x4{0, 0, 0, 0};
            if (left) {
                const int j = __builtin_ctzll(left);
                left &= left - 1;
                const int64_t row = __builtin_amdgcn_readlane(c.row, j);
                w[i] = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(c.w), j));
                v[i] = load_stream(reinterpret_cast<const u32x4*>(y + row * K + el));
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float f[8];
            unpack8(v[i], f);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                acc[q] = __builtin_fmaf(w[i], f[q], acc[q]);
        }
    }
    if (in)
        store_stream(reinterpret_cast<u32x4*>(out + t * K + e0), pack8(acc));
}

// kWaves waves per token: wave w takes the 512-element pieces w, w + kWaves, ... of its rows.
template <int kWaves>
__global__ __launch_bounds__(kWaves > 4 ? 64 * kWaves : kThreads) void combine_backward_kernel(
    const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y, const int32_t* __restrict__ pos,
    const float* __restrict__ weights, uint16_t* __restrict__ dy, float* __restrict__ dweights, int64_t n_tokens,
    int k, int64_t M_cap, int64_t K)
{
    constexpr int kTokens = kWaves > 4 ? 1 : kThreads / 64 / kWaves;      // tokens of a workgroup
    __shared__ float part[kTokens][kWaves][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = wave % kWaves, tok = wave / kWaves;
    const int64_t t = (int64_t)blockIdx.x * kTokens + tok;
    if (t < n_tokens) {
        const Choices c = choices_of(pos, weights, t, k, M_cap);
        part[tok][sub][lane] = 0.0f;              // the choices without a row keep it
        wave_lds_order();                         // (the sums come from lane 0)
        for (uint64_t left = c.live; left;) {
            int64_t row[kBatch];
            float w[kBatch], dot[kBatch] = {};
            int n = 0;
            const uint64_t these = left;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                row[i] = 0;
                w[i] = 0.0f;
                if (left) {
                    const int j = __builtin_ctzll(left);
                    left &= left - 1;
                    row[i] = __builtin_amdgcn_readlane(c.row, j);
                    w[i] = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(c.w), j));
                    ++n;
                }
            }
            for (int64_t e0 = 512 * sub + 8 * lane; e0 < K; e0 += 512 * kWaves) {
                float d[8];
                unpack8(*reinterpret_cast<const u32x4*>(dout + t * K + e0), d);
                u32x4 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (i < n)
                        v[i] = load_stream(reinterpret_cast<const u32x4*>(y + row[i] * K + e0));
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (i < n) {
                        float f[8], o[8];
                        unpack8(v[i], f);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            dot[i] = __builtin_fmaf(d[q], f[q], dot[i]);
                            o[q] = w[i] * d[q];
                        }
                        store_stream(reinterpret_cast<u32x4*>(dy + row[i] * K + e0), pack8(o));
                    }
            }
            uint64_t at = these;
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (i < n) {
                    const int j = __builtin_ctzll(at);
                    at &= at - 1;
                    const float s = wave_sum(dot[i]);
                    if (lane == 0)
                        part[tok][sub][j] = s;
                }
        }
    }
    __syncthreads();
    if (t < n_tokens && sub == 0 && lane < k) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            s += part[tok][w][lane];
        dweights[t * k + lane] = s;
    }
}

hipError_t launch_combine(const uint16_t* y, const int32_t* pos, const float* weights, const uint16_t* base,
                          uint16_t* out, int64_t T, int32_t k, int64_t M_cap, int64_t K, hipStream_t stream)
{
    uint32_t units = (uint32_t)((K + 511) / 512);
    const int64_t grid = (T * units + kThreads / 64 - 1) / (kThreads / 64);
    if (grid > 0x7FFFFFFF)
        return hipErrorInvalidValue;
    int kk = k;
    int64_t t = T, cap = M_cap, w = K;
    void* args[] = {(void*)&y, (void*)&pos, (void*)&weights, (void*)&base, (void*)&out, (void*)&t,
                    (void*)&kk, (void*)&cap, (void*)&w, (void*)&units};
    return launch_kernel((const void*)combine_kernel, dim3((unsigned)grid), dim3(kThreads), args, stream);
}

hipError_t launch_combine_backward(const uint16_t* dout, const uint16_t* y, const int32_t* pos, const float* weights,
                                   uint16_t* dy, float* dweights, int64_t T, int32_t k, int64_t M_cap, int64_t K,
                                   hipStream_t stream)
{
    // waves per token as far as the row has pieces for them, more for few tokens (64 tokens x
    // 7168, 8 choices: 8.7 us with 16, 11.0 with 4; 4099 tokens x 2048, 6 choices: 40.8 with 4,
    // 48.0 with 1; 8192 x 7168, 8 choices: 380 with 4, 391 with 1)
    const int waves = K <= 512 ? 1 : T < 256 && K > 2048 ? 16 : 4;
    const int64_t per = waves == 1 ? kThreads / 64 : 1;
    const int64_t grid = (T + per - 1) / per;
    if (grid > 0x7FFFFFFF)
        return hipErrorInvalidValue;
    int kk = k;
    int64_t t = T, cap = M_cap, w = K;
    void* args[] = {(void*)&dout, (void*)&y, (void*)&pos, (void*)&weights, (void*)&dy, (void*)&dweights,
                    (void*)&t, (void*)&kk, (void*)&cap, (void*)&w};
    const void* kernel = waves == 1   ? (const void*)combine_backward_kernel<1>
                         : waves == 4 ? (const void*)combine_backward_kernel<4>
                                      : (const void*)combine_backward_kernel<16>;
    return launch_kernel(kernel, dim3((unsigned)grid), dim3((unsigned)(waves > 4 ? 64 * waves : kThreads)), args,
                         stream);
}

}  // namespace mxfp4
