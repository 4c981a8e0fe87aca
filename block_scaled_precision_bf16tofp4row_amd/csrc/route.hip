// route.hip -- routing of tokens to experts, and its gradient.
//
// Forward, for the logits l[t, 0..E) of token t:
//     s_e = softmax(l)_e  or  1 / (1 + exp(-l_e));   c_e = s_e + bias_e (selection only)
//     a group's value: the sum of its group_best largest c; the topk_group best groups stay
//     ids = the k largest c of the groups that stay (equal values: the lower index first)
//     w_j = scale * s[ids_j] / (sum_i s[ids_i] + 1e-20), or scale * s[ids_j]
// Backward, with D = sum_i s_i + 1e-20 over the selected experts:
//     ds_j = scale * (dw_j - sum_i dw_i s_i / D) / D, or scale * dw_j
//     softmax: dl_e = s_e (ds_e - sum_j ds_j s_j), ds_e = 0 where e is not selected
//     sigmoid: dl_e = s_e (1 - s_e) ds_e
// All of it in FP32; the logits are read once (16-byte loads where the rows allow them).
//
// Selection works on order keys: the FP32 bits of c made monotone as unsigned integers,
// NaN below every number, and 0 for what is excluded, so that a comparison is one integer
// maximum and any input gives k distinct valid indices.
#include "strips.h"

namespace mxfp4 {

namespace {

constexpr int kMaxRouteV = 32;                    // experts per lane at most

// exp(x) in FP32 to about 2 units in the last place: 2^(x log2 e) with the product's
// rounding error put back (x log2 e carries an absolute error of |x| 2^-24 otherwise).
__device__ __forceinline__ float exp_f32(float x)
{
    constexpr float kHi = 1.44269502162933349609375f;        // log2 e, rounded to FP32
    constexpr float kLo = 1.9259629911e-8f;                // log2 e - kHi
    constexpr float kLn2 = 0.6931471805599453f;
    const float t = x * kHi;
    const float e = __builtin_amdgcn_exp2f(t);
    const float lo = __builtin_fmaf(x, kHi, -t) + x * kLo;
    const float r = __builtin_fmaf(e, lo * kLn2, e);
    return __builtin_isfinite(r) ? r : e;         // exp(+-inf), exp(NaN) as they are
}

__device__ __forceinline__ float sigmoid_f32(float x) { return 1.0f / (1.0f + exp_f32(-x)); }

// FP32 -> order key: larger key, larger value; NaN gives 1 (below -inf), never 0.
__device__ __forceinline__ uint32_t order_key(float c)
{
    c += 0.0f;                                    // -0 and +0 are equal
    const uint32_t b = __float_as_uint(c);
    const uint32_t k = (int32_t)b < 0 ? ~b : b | 0x80000000u;
    return c == c ? k : 1u;
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return k <= 1u ? __uint_as_float(0x7FC00000u) : __uint_as_float((int32_t)k < 0 ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        v += __shfl_xor(v, d, 64);
    return v;
}
__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, d, 64));
    return uniform(v);
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// What a softmax row is normalised by: p_e = exp(l_e - m) * inv.  A row of -inf only has
// p = 0 everywhere; a row with NaN or +inf has NaN everywhere.
struct RowNorm {
    float m, inv;
};
__device__ __forceinline__ float softmax_of(float l, RowNorm n) { return exp_f32(l - n.m) * n.inv; }
__device__ __forceinline__ RowNorm row_norm(float m, float sum)
{
    RowNorm n;
    n.m = m == -__builtin_inff() ? 0.0f : m;
    n.inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    return n;
}

}  // namespace

// One wave per token.  Each group has L lanes (64 / n_group rounded down to a power of
// two) and each of them VPL consecutive experts of it, so lane order is expert order
// and what a group needs is exchanged inside its lanes.
template <int VPL, typename T>
__global__ __launch_bounds__(kThreads) void route_kernel(
    const T* __restrict__ logits, const float* __restrict__ bias, const uint8_t* __restrict__ row_mask,
    int32_t* __restrict__ ids, float* __restrict__ weights, int64_t n_tokens, int E, int n_group, int topk_group,
    int group_best, int k, int sigmoid, int renorm, float scale, int L)
{
    __shared__ float s_lds[kThreads / 64][64 * VPL];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + wave;
    if (t >= n_tokens)
        return;
    const int gs = E / n_group;
    const int g = lane / L, r = lane & (L - 1);
    const int e0 = g * gs + r * VPL;              // the lane's first expert
    const int nv = g < n_group ? min(VPL, gs - r * VPL) : 0;
    const T* const row = logits + t * E;

    float s[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        s[i] = i < nv ? load_logit(row + e0 + i) : -__builtin_inff();
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            s[i] = sigmoid_f32(s[i]);
    } else {
        float m = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            m = fmaxf(m, s[i]);
        m = wave_max(m);
        const float m0 = m == -__builtin_inff() ? 0.0f : m;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            s[i] = exp_f32(s[i] - m0);
            sum += s[i];
        }
        const RowNorm n = row_norm(m, wave_sum(sum));
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            s[i] *= n.inv;
    }
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        key[i] = i < nv ? order_key(s[i] + (bias ? bias[e0 + i] : 0.0f)) : 0u;
        s_lds[wave][lane * VPL + i] = s[i];
    }
    if (topk_group < n_group) {
        uint32_t k1 = 0, k2 = 0;                  // the two largest keys of the group
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            k2 = max(k2, min(k1, key[i]));
            k1 = max(k1, key[i]);
        }
        for (int d = 1; d < L; d <<= 1) {
            const uint32_t o1 = (uint32_t)__shfl_xor((int)k1, d, 64), o2 = (uint32_t)__shfl_xor((int)k2, d, 64);
            k2 = max(max(k2, o2), min(k1, o1));
            k1 = max(k1, o1);
        }
        const float v = group_best == 2 ? key_value(k1) + key_value(k2) : key_value(k1);
        const uint32_t gk = order_key(v);
        int rank = 0;
        for (int h = 0; h < n_group; ++h) {
            const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)gk, h * L);
            rank += o > gk || (o == gk && h < g);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            key[i] = rank < topk_group ? key[i] : 0u;
    }
    int mine = 0;                                 // lane j: place of selection j in s_lds
    for (int j = 0; j < k; ++j) {
        uint32_t lm = key[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i)
            lm = max(lm, key[i]);
        const uint32_t best = wave_max_u32(lm);
        const int src = __builtin_ctzll(__ballot(lm == best));
        int slot = 0;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
            slot = key[i] == best ? i : slot;
        slot = __builtin_amdgcn_readlane(slot, src);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            key[i] = lane == src && i == slot ? 0u : key[i];
        mine = lane == j ? src * VPL + slot : mine;
    }
    const float sj = lane < k ? s_lds[wave][mine] : 0.0f;
    float w = scale * sj;
    if (renorm)
        w = scale * (sj / (wave_sum(sj) + 1e-20f));
    const int from = mine / VPL;
    int e = (from / L) * gs + (from & (L - 1)) * VPL + mine % VPL;
    if (row_mask && !row_mask[t]) {
        e = -1;
        w = 0.0f;
    }
    if (lane < k) {
        ids[t * k + lane] = e;
        weights[t * k + lane] = w;
    }
}

// One wave per token; lane j < k holds selection j.  The selected experts' ds are placed in
// a row of LDS (zero elsewhere), from which every lane takes its experts'.
template <typename T>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ dweights,
    T* __restrict__ dlogits, int64_t n_tokens, int E, int k, int sigmoid, int renorm, float scale)
{
    constexpr int kV = 16;                        // E <= 1024
    __shared__ float ds_lds[kThreads / 64][64 * kV];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + wave;
    if (t >= n_tokens)
        return;
    const T* const row = logits + t * E;
    float p[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int e = i * 64 + lane;
        p[i] = e < E ? load_logit(row + e) : -__builtin_inff();
        if (e < E)
            ds_lds[wave][e] = 0.0f;
    }
    RowNorm n{0.0f, 1.0f};
    if (!sigmoid) {
        float m = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < kV; ++i)
            m = fmaxf(m, p[i]);
        m = wave_max(m);
        const float m0 = m == -__builtin_inff() ? 0.0f : m;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i)
            sum += exp_f32(p[i] - m0);
        n = row_norm(m, wave_sum(sum));
    }
    int id = -1;
    float dw = 0.0f, sj = 0.0f;
    if (lane < k) {
        id = ids[t * k + lane];
        if ((uint32_t)id < (uint32_t)E) {
            dw = dweights[t * k + lane];
            const float l = load_logit(row + id);
            sj = sigmoid ? sigmoid_f32(l) : softmax_of(l, n);
        } else {
            id = -1;
        }
    }
    float ds = scale * dw;
    if (renorm) {
        const float D = wave_sum(sj) + 1e-20f;
        ds = scale * ((dw - wave_sum(dw * sj) / D) / D);
    }
    if (id >= 0)
        ds_lds[wave][id] = ds;
    else
        ds = 0.0f;
    const float dot = sigmoid ? 0.0f : wave_sum(ds * sj);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int e = i * 64 + lane;
        if (e < E) {
            const float d = ds_lds[wave][e];
            const float q = sigmoid ? sigmoid_f32(p[i]) : softmax_of(p[i], n);
            const float out = sigmoid ? d * (q * (1.0f - q)) : q * (d - dot);
            if constexpr (sizeof(T) == 4)
                dlogits[t * E + e] = out;
            else
                dlogits[t * E + e] = __builtin_bit_cast(uint16_t, (__bf16)out);
        }
    }
}

template <typename T>
static const void* route_kernel_for(int vpl)
{
    switch (vpl) {
    case 1: return (const void*)route_kernel<1, T>;
    case 2: return (const void*)route_kernel<2, T>;
    case 4: return (const void*)route_kernel<4, T>;
    case 8: return (const void*)route_kernel<8, T>;
    case 16: return (const void*)route_kernel<16, T>;
    default: return (const void*)route_kernel<kMaxRouteV, T>;
    }
}

hipError_t launch_route(const void* logits, bool f32, const float* bias, const uint8_t* row_mask, int32_t* ids,
                        float* weights, int64_t T, int32_t E, int32_t n_group, int32_t topk_group,
                        int32_t group_best, int32_t k, bool sigmoid, bool renorm, float scale, hipStream_t stream)
{
    const int64_t grid = (T + kThreads / 64 - 1) / (kThreads / 64);
    if (grid > 0x7FFFFFFF)
        return hipErrorInvalidValue;
    int L = 1;
    while (2 * L * n_group <= 64)
        L *= 2;
    const int need = (E / n_group + L - 1) / L;   // experts per lane
    int vpl = 1;
    while (vpl < need)
        vpl *= 2;
    if (vpl > kMaxRouteV)
        return hipErrorInvalidValue;
    int64_t t = T;
    int e = E, ng = n_group, tg = topk_group, gb = group_best, kk = k, sg = sigmoid, rn = renorm;
    float sc = scale;
    void* args[] = {(void*)&logits, (void*)&bias, (void*)&row_mask, (void*)&ids, (void*)&weights, (void*)&t, (void*)&e,
                    (void*)&ng, (void*)&tg, (void*)&gb, (void*)&kk, (void*)&sg, (void*)&rn, (void*)&sc, (void*)&L};
    return launch_kernel(f32 ? route_kernel_for<float>(vpl) : route_kernel_for<uint16_t>(vpl), dim3((unsigned)grid),
                         dim3(kThreads), args, stream);
}

hipError_t launch_route_backward(const void* logits, bool f32, const int32_t* ids, const float* dweights,
                                 void* dlogits, int64_t T, int32_t E, int32_t k, bool sigmoid, bool renorm,
                                 float scale, hipStream_t stream)
{
    const int64_t grid = (T + kThreads / 64 - 1) / (kThreads / 64);
    if (grid > 0x7FFFFFFF)
        return hipErrorInvalidValue;
    int64_t t = T;
    int e = E, kk = k, sg = sigmoid, rn = renorm;
    float sc = scale;
    void* args[] = {(void*)&logits, (void*)&ids, (void*)&dweights, (void*)&dlogits, (void*)&t, (void*)&e,
                    (void*)&kk, (void*)&sg, (void*)&rn, (void*)&sc};
    return launch_kernel(f32 ? (const void*)route_backward_kernel<float> : (const void*)route_backward_kernel<uint16_t>,
                         dim3((unsigned)grid), dim3(kThreads), args, stream);
}

}  // namespace mxfp4
