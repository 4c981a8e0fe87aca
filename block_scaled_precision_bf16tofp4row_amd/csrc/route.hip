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
//     sigmoid: dl_e = s_e (1 - s_e) ds_e, s (1 - s) as e / (1 + e)^2 with e = exp(-|l|)
// All of it in FP32; the logits are read once (16-byte loads where the rows allow them).
//
// Selection works on order keys: the FP32 bits of c made monotone as unsigned integers,
// NaN below every number, and 0 for what is excluded, so that a comparison is one integer
// maximum and any input gives k distinct valid indices.
//
// What bounds it: 32768 tokens x 256 experts in 8 groups, FP32 logits, 8 choices: 11.4-12.4 us
// for 36 MB, which a copy moves in 7.0; the vector unit is busy for 80 % of the time (600
// instructions per four tokens, half of them the scores and keys, a fifth the sort), with half
// the bytes (BF16, softmax) it is 9.8 us.  32768 x 64, softmax: 5.5 us.  Few tokens are a
// launch: 3.5 us for one, 4.0 for 128.  The gradient is its bytes: 16384 x 256, FP32, softmax:
// 7.9 us for 35 MB (6.8 copied), sigmoid, which reads the chosen logits only: 6.2.
#include "lanes.h"

namespace mxfp4 {

namespace {

constexpr int kMaxRouteV = 32;                    // experts per lane at most

constexpr float kLog2eHi = 1.44269502162933349609375f;       // log2 e, rounded to FP32
constexpr float kLog2eLo = 1.9259629911e-8f;                 // and the rest of it

// exp(x + dx) in FP32 to about 2 units in the last place, for x <= 0 and dx far below x:
// 2^(x log2 e) with the product's rounding error put back (x log2 e carries an absolute error
// of |x| 2^-24 otherwise).  Where x log2 e is -inf, and the result 0, the correction is
// infinite or NaN: the median makes it finite (it is below 2^-13 elsewhere).
__device__ __forceinline__ float exp_f32(float x, float dx = 0.0f)
{
    constexpr float kLn2 = 0.6931471805599453f;
    const float t = x * kLog2eHi;
    const float e = __builtin_amdgcn_exp2f(t);
    const float lo = __builtin_fmaf(x, kLog2eLo, __builtin_fmaf(x, kLog2eHi, -t));
    return __builtin_fmaf(e, __builtin_amdgcn_fmed3f(__builtin_fmaf(lo, kLn2, dx), -1.0f, 1.0f), e);
}

// The forward pass takes exp of every logit without that correction, for the order keys and a
// softmax row's sum, and forms the scores of the chosen anew for their weights.  A softmax
// row's terms are off by |x| 2^-24 and the instruction's unit, to either side: in the sum that
// weighs |x| e^x, a few 2^-24 at most (with the correction 32768 x 256, BF16: 10.5 us for 9.8).
__device__ __forceinline__ float exp_row(float x)
{
    return __builtin_amdgcn_exp2f(__builtin_fmaf(x, kLog2eHi, x * kLog2eLo));
}
// A sigmoid's key: off by |x| (2^-24 + 1.4e-8) of itself, in part to one side, and the
// exponential's and the reciprocal's unit each.  It rises with x, so it decides like the exact
// score but for what differs by less than that beside a bias or in a group's sum.
__device__ __forceinline__ float sigmoid_key(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2eHi));
}
// The sigmoid and its derivative.  From e = exp(-|x|) neither is a difference of nearly equal
// numbers: s (1 - s) of the rounded s has 4 bits left at x = 16, where it is as confident as
// the experts that are chosen, and none from 17 on.
struct Sigmoid {
    float s, ds;
};
__device__ __forceinline__ Sigmoid sigmoid_f32(float x)
{
    const float e = exp_f32(-__builtin_fabsf(x)), d = 1.0f + e;
    float r = __builtin_amdgcn_rcpf(d);           // 1 / d, d in [1, 2]: one Newton step rounds it
    r = __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r);
    return {x < 0.0f ? e * r : r, e * r * r};
}

// FP32 -> order key: larger key, larger value.  Numbers take 0x00FFFFFE (-inf) to 0xFFFFFFFF
// (+inf); the sum that puts +inf there lets every NaN wrap to less than -inf, and the maximum
// makes them one.  No key is 0.  (No sum of a score, which is +0 or more, and a bias is -0.)
constexpr uint32_t kKeyOffset = 0x807FFFFFu, kKeyNaN = 0x00FFFFFDu;
__device__ __forceinline__ uint32_t order_key(float c)
{
    const uint32_t b = __float_as_uint(c);
    return max((b ^ ((uint32_t)((int32_t)b >> 31) & 0x7FFFFFFFu)) + kKeyOffset, kKeyNaN);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    const uint32_t b = k - kKeyOffset;
    return __uint_as_float(k <= kKeyNaN ? 0x7FC00000u : b ^ ((uint32_t)((int32_t)b >> 31) & 0x7FFFFFFFu));
}

// What lane ^ D holds, for a value that is the same in every aligned run of D lanes.
template <int D>
__device__ __forceinline__ uint32_t across(uint32_t v)
{
    if constexpr (D == 1)
        return dpp<kQuadSwap1>(v);
    else if constexpr (D == 2)
        return dpp<kQuadSwap2>(v);
    else if constexpr (D == 4)
        return dpp<kRowHalfMirror>(v);
    else if constexpr (D == 8)
        return dpp<kRowMirror>(v);
    else
        return (uint32_t)__shfl_xor((int)v, D, 64);
}
// The two largest keys of the 1 << l_log lanes of a group, from each lane's two largest.
template <int D = 1>
__device__ __forceinline__ void group_top2(uint32_t& k1, uint32_t& k2, int l_log)
{
    if constexpr (D < 64) {
        if (D >> l_log)
            return;                               // (uniform)
        const uint32_t o1 = across<D>(k1), o2 = across<D>(k2);
        k2 = max(max(k2, o2), min(k1, o1));
        k1 = max(k1, o1);
        group_top2<2 * D>(k1, k2, l_log);
    }
}

// value[lane] = mask has the lane ? 0 : value, the mask on the scalar unit.
__device__ __forceinline__ void clear_lanes(uint32_t& v, uint64_t mask)
{
    asm("v_cndmask_b32 %0, %0, 0, %1" : "+v"(v) : "s"(mask));
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
typedef float f32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ f32x4 load_logit4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load_logit4(const uint16_t* p)
{
    const u32x2 u = *reinterpret_cast<const u32x2*>(p);
    return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                 __uint_as_float(u.y & 0xFFFF0000u)};
}

// What a softmax row is normalised by: p_e = exp(l_e - m) * inv.  A row of -inf only has
// p = 0 everywhere; a row with NaN or +inf has NaN everywhere.
struct RowNorm {
    float m, inv;
};
// One of its scores, with what l - m loses put back (half a unit of the difference: 4e-6 of the
// score at 80 below the maximum).  In the row's sum such terms weigh nothing and go without.
__device__ __forceinline__ float softmax_of(float l, RowNorm n)
{
    const float d = l - n.m, b = d - l;           // (the exact error of a difference, after Knuth)
    const float err = (l - (d - b)) - (n.m + b);
    return exp_f32(d, err) * n.inv;
}
// The maximum from its key (0 for a row of -inf or NaN only), the factor from the sum (NaN if
// a logit is NaN, which the maximum leaves out).
__device__ __forceinline__ float norm_top(uint32_t key)
{
    const float m = key_value(key);
    return m == -__builtin_inff() || !(m == m) ? 0.0f : m;
}
__device__ __forceinline__ float norm_inv(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }
// The norm of a row spread over a wave, and its scores in place of the logits.
template <int V>
__device__ __forceinline__ RowNorm softmax_row(float (&l)[V])
{
    float top = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i)
        top = fmaxf(top, l[i]);
    RowNorm n;
    n.m = norm_top(wave_max(order_key(top)));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        sum += l[i] = exp_row(l[i] - n.m);
    n.inv = norm_inv(wave_sum(sum));
#pragma unroll
    for (int i = 0; i < V; ++i)
        l[i] *= n.inv;
    return n;
}

}  // namespace

// One wave per token, several in turn.  Each group has L = 1 << l_log lanes (64 / n_group
// rounded down to a power of two) and each of them VPL consecutive experts of it, so lane
// order is expert order and what a group needs is exchanged inside its lanes.  A selection
// is one wave maximum (six DPP steps); the lane and slot that hold it are found on the
// scalar unit from one ballot per slot.  VEC: VPL is a multiple of 4, groups are too and
// rows aligned, so a lane's logits are 16-byte (BF16: 8-byte) loads.
// The selections, one after the other, are its time: 32768 tokens x 384 with 8 choices 44 us
// for 52 MB (10.3 copied), x 512 with 10 choices 53 (13.7), x 160 in 8 groups with 6 choices
// 28 (4.4), x 32 in 8 groups with 8 choices 16 (1.2).
template <int VPL, bool VEC, typename T>
__global__ __launch_bounds__(kThreads) void route_kernel(
    const T* __restrict__ logits, const float* __restrict__ bias, const uint8_t* __restrict__ row_mask,
    int32_t* __restrict__ ids, float* __restrict__ weights, int64_t n_tokens, int E, int n_group, int gs,
    int topk_group, int group_best, int k, int sigmoid, int renorm, float scale, int l_log)
{
    __shared__ __attribute__((aligned(16))) float l_lds[kThreads / 64][64 * VPL];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t step = (int64_t)gridDim.x * (kThreads / 64);
    int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + wave;
    if (t >= n_tokens)
        return;
    const int g = lane >> l_log, r = lane & ((1 << l_log) - 1);
    const int e0 = g * gs + r * VPL;              // the lane's first expert
    const int nv = g < n_group ? gs - r * VPL : 0;       // the experts it has, at most VPL of them

    // (slots without an expert read another one's)
    auto load_row = [&](float (&v)[VPL], const auto* row) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < VPL; i += 4) {
                const f32x4 q = load_logit4(row + (i < nv ? e0 + i : 0));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[i + j] = q[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                v[i] = load_logit(row + (i < nv ? e0 + i : 0));
        }
    };
    float b[VPL] = {}, next[VPL];
    if (bias)
        load_row(b, bias);
    load_row(next, logits + t * E);
    for (; t < n_tokens; t += step) {
        float s[VPL];
        RowNorm n{0.0f, 1.0f};
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            l_lds[wave][lane * VPL + i] = s[i] = next[i];
        if (t + step < n_tokens)
            load_row(next, logits + (t + step) * E);
        if (sigmoid) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                s[i] = sigmoid_key(s[i]);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                s[i] = i < nv ? s[i] : -__builtin_inff();
            n = softmax_row(s);
        }
        uint32_t key[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            key[i] = order_key(s[i] + b[i]) & (i < nv ? ~0u : 0u);
        if (topk_group < n_group) {
            uint32_t k1 = 0, k2 = 0;              // the two largest keys of the lane, then of the group
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                k2 = max(k2, min(k1, key[i]));
                k1 = max(k1, key[i]);
            }
            group_top2(k1, k2, l_log);
            const float v = group_best == 2 ? key_value(k1) + key_value(k2) : key_value(k1);
            const uint32_t gk = order_key(v);
            int rank = 0;
            for (int h = 0; h < n_group; ++h) {
                const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)gk, h << l_log);
                rank += o > gk - (h < g);         // a group before this one wins ties (no key is 0)
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                key[i] = rank < topk_group ? key[i] : 0u;
        }
        int mine = 0;                             // lane j: place of selection j in l_lds
        for (int j = 0; j < k; ++j) {
            uint32_t lm = key[0];
#pragma unroll
            for (int i = 1; i < VPL; ++i)
                lm = max(lm, key[i]);
            const uint32_t best = wave_max(lm);
            // the first lane that holds it, and its first slot that does, on the scalar unit
            uint64_t has[VPL], any = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                has[i] = __ballot(key[i] == best);
                any |= has[i];
            }
            const uint64_t first = any & (0 - any);
            uint32_t slots = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                slots |= (has[i] & first) != 0 ? 1u << i : 0u;
            const uint32_t slot = slots & (0 - slots);
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                clear_lanes(key[i], slot == 1u << i ? first : 0);
            const int at = (int)__builtin_ctzll(any) * VPL + __builtin_ctz(slots);
            mine = lane == j ? at : mine;
        }
        wave_lds_order();
        const float l = l_lds[wave][mine];        // (of every lane: place 0 past the choices)
        wave_lds_order();                         // the next token's logits take its place
        float sj = 0.0f;
        if (lane < k)
            sj = sigmoid ? sigmoid_f32(l).s : softmax_of(l, n);
        float w = scale * sj;
        if (renorm)
            w = scale * (sj / (wave_sum(sj) + 1e-20f));
        const int from = mine / VPL;
        int e = (from >> l_log) * gs + (from & ((1 << l_log) - 1)) * VPL + mine % VPL;
        if (row_mask && !row_mask[t]) {
            e = -1;
            w = 0.0f;
        }
        if (lane < k) {
            ids[t * k + lane] = e;
            weights[t * k + lane] = w;
        }
    }
}

// ---- four tokens per wave -------------------------------------------------------------
// Up to 256 experts and 8 choices: 16 lanes (a DPP row) per token, VPL consecutive experts
// per lane.  A candidate is one number, the bits of a double in [2, 4) with the order key in
// the top 32 bits of its mantissa and the expert below (the complements of its lane and of
// its slot there, so that the lower expert is the larger number): no two are equal, the larger
// one is the better choice, and v_max_f64 / v_min_f64 sort them without carrying an index
// along.  Each lane sorts its candidates (the best 8 of them), the groups are ranked on the
// lists' heads, then k times the row's best head is taken (four DPP steps) and its lane moves
// on in its list, which lies in LDS.  Against one token per wave: 32768 x 256 in 8 groups 12.8
// and 31.5 us, 32768 x 64 5.6 and 12.7, 128 x 256 4.2 both.

__device__ __forceinline__ double f64_max(double a, double b)
{
    double d;                                     // (fmax would first quiet its operands)
    asm("v_max_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}
__device__ __forceinline__ double f64_min(double a, double b)
{
    double d;
    asm("v_min_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}
__device__ __forceinline__ double candidate(uint32_t key, uint32_t low)
{
    const uint32_t hi = __builtin_amdgcn_alignbit(0x400u, key, 12), lo = key << 20 | low;
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ uint32_t key_of(double c)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, c);
    return __builtin_amdgcn_alignbit((uint32_t)(u >> 32), (uint32_t)u, 20);
}
__device__ __forceinline__ double with_low(double c, uint32_t low)
{
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, c) | low);
}
__device__ __forceinline__ void order2(double& a, double& b)
{
    const double hi = f64_max(a, b);
    b = f64_min(a, b);
    a = hi;
}
__device__ __forceinline__ void sort4(double* v)
{
    order2(v[0], v[1]), order2(v[2], v[3]);
    order2(v[0], v[2]), order2(v[1], v[3]);
    order2(v[1], v[2]);
}
__device__ __forceinline__ void sort8(double* v)          // Batcher's odd-even merge of two sorted halves
{
    sort4(v), sort4(v + 4);
    order2(v[0], v[4]), order2(v[1], v[5]), order2(v[2], v[6]), order2(v[3], v[7]);
    order2(v[2], v[4]), order2(v[3], v[5]);
    order2(v[1], v[2]), order2(v[3], v[4]), order2(v[5], v[6]);
}
// The best min(V, 8) of V candidates, in order, in the first places.
template <int V>
__device__ __forceinline__ void sort_best(double (&v)[V])
{
    if constexpr (V == 4) {
        sort4(v);
    } else if constexpr (V == 8) {
        sort8(v);
    } else {
        sort8(v), sort8(v + 8);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = f64_max(v[i], v[15 - i]);      // the best 8, a bitonic sequence
        order2(v[0], v[4]), order2(v[1], v[5]), order2(v[2], v[6]), order2(v[3], v[7]);
        order2(v[0], v[2]), order2(v[1], v[3]), order2(v[4], v[6]), order2(v[5], v[7]);
        order2(v[0], v[1]), order2(v[2], v[3]), order2(v[4], v[5]), order2(v[6], v[7]);
    }
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32 | dpp<CTRL>((uint32_t)u));
}
__device__ __forceinline__ double row_best(double v)
{
    v = f64_max(v, dpp<kQuadSwap1>(v));
    v = f64_max(v, dpp<kQuadSwap2>(v));
    v = f64_max(v, dpp<kRowHalfMirror>(v));
    return f64_max(v, dpp<kRowMirror>(v));
}
// How many of the row's other groups come before this lane's: the groups have L lanes each
// and fill the row, so rotations by L lanes show each of them.
template <int L, int N = L>
__device__ __forceinline__ int group_rank(uint32_t gk, uint32_t g)
{
    if constexpr (N < 16) {
        constexpr int kRor = 0x120 + N;
        const uint32_t before = dpp<kRor>(g) < g;          // it wins ties (no key is 0)
        return (dpp<kRor>(gk) > gk - before) + group_rank<L, N + L>(gk, g);
    }
    return 0;
}

template <int VPL, bool VEC, typename T>
__global__ __launch_bounds__(kThreads) void route_quad_kernel(
    const T* __restrict__ logits, const float* __restrict__ bias, const uint8_t* __restrict__ row_mask,
    int32_t* __restrict__ ids, float* __restrict__ weights, int64_t n_tokens, int E, int n_group, int gs,
    int topk_group, int group_best, int k, int sigmoid, int renorm, float scale, int l_log)
{
    constexpr int kList = VPL < 8 ? VPL : 8;
    __shared__ double list[kThreads / 64][kList + 1][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15;                      // lane of the row
    const int64_t t = ((int64_t)blockIdx.x * (kThreads / 64) + wave) * 4 + (lane >> 4);
    if (t - (lane >> 4) >= n_tokens)
        return;
    const int e0 = r * VPL;                       // the lane's first expert
    const int nv = E - e0;                        // the experts it has, at most VPL of them
    const T* const row = logits + min(t, n_tokens - 1) * E;

    // (slots without an expert read another one's, rows without a token the last one's)
    auto load_row = [&](float (&v)[VPL], const auto* from) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < VPL; i += 4) {
                const f32x4 q = load_logit4(from + (i < nv ? e0 + i : 0));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[i + j] = q[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                v[i] = load_logit(from + (i < nv ? e0 + i : 0));
        }
    };
    float s[VPL], b[VPL] = {};
    RowNorm n{0.0f, 1.0f};
    load_row(s, row);
    if (bias)
        load_row(b, bias);
    const bool chosen = row_mask == nullptr || row_mask[min(t, n_tokens - 1)] != 0;
    list[wave][kList][lane] = 0.0;                // below every candidate
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            s[i] = sigmoid_key(s[i]);
    } else {
        float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            s[i] = i < nv ? s[i] : -__builtin_inff();
            top = fmaxf(top, s[i]);
        }
        n.m = norm_top(row_max(order_key(top)));
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            sum += s[i] = exp_row(s[i] - n.m);
        n.inv = norm_inv(row_sum(sum));
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            s[i] *= n.inv;
    }
    double c[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        c[i] = candidate(order_key(s[i] + b[i]), (uint32_t)(VPL - 1 - i));
    if (E < 16 * VPL) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            c[i] = i < nv ? c[i] : candidate(0, 0);
    }
    sort_best(c);
#pragma unroll
    for (int i = 0; i < kList; ++i)
        c[i] = with_low(c[i], (uint32_t)(15 - r) * VPL);       // (VPL is a power of two)
#pragma unroll
    for (int i = 1; i < kList; ++i)
        list[wave][i][lane] = c[i];
    double head = c[0];
    if (topk_group < n_group) {
        uint32_t k1 = key_of(c[0]), k2 = key_of(c[1]);
        group_top2(k1, k2, l_log);
        const uint32_t gk = order_key(group_best == 2 ? key_value(k1) + key_value(k2) : key_value(k1));
        const uint32_t g = (uint32_t)r >> l_log;
        const int rank = l_log == 0   ? group_rank<1>(gk, g)
                         : l_log == 1 ? group_rank<2>(gk, g)
                         : l_log == 2 ? group_rank<4>(gk, g)
                                      : group_rank<8>(gk, g);
        head = rank < topk_group ? head : 0.0;    // a lane's experts are of one group
    }
    const double* rest = &list[wave][1][lane];
    uint32_t mine = 0;                            // lane j of the row: the low bits of choice j
    for (int j = 0; j < k; ++j) {
        const double best = row_best(head);
        if (__builtin_bit_cast(uint64_t, head) == __builtin_bit_cast(uint64_t, best)) {
            head = *rest;
            rest += 64;
        }
        mine = r == j ? (uint32_t)__builtin_bit_cast(uint64_t, best) : mine;
    }
    const int e = 16 * VPL - 1 - (int)(mine & (16 * VPL - 1));
    float sj = 0.0f;                              // its score once more, from the cached logit
    if (r < k) {
        const float l = load_logit(row + e);
        sj = sigmoid ? sigmoid_f32(l).s : softmax_of(l, n);
    }
    float w = scale * sj;
    if (renorm)
        w = scale * (sj / (row_sum(sj) + 1e-20f));
    if (t < n_tokens && r < k) {
        ids[t * k + r] = chosen ? e : -1;
        weights[t * k + r] = chosen ? w : 0.0f;
    }
}

// ---- backward ---------------------------------------------------------------------------

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) { return LANES == 16 ? row_sum(v) : wave_sum(v); }
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) { return LANES == 16 ? row_max(v) : wave_max(v); }

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void store_logit4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store_logit4(uint16_t* p, f32x4 v)
{
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    const bf16x4 b = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    *reinterpret_cast<u32x2*>(p) = __builtin_bit_cast(u32x2, b);
}

// LANES lanes per token, 4 Q experts per lane in runs of four (LANES x 4 consecutive experts
// per load); lane j < k holds selection j.  The selected experts' ds are placed in a row of
// LDS that is zero elsewhere, from which every lane takes its experts'.  Reading and writing
// the logits is what bounds it (16384 tokens x 256 experts, FP32: 34.6 MB).
template <int LANES, int Q, bool VEC, bool SIGMOID, typename T>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ dweights,
    T* __restrict__ dlogits, int64_t n_tokens, int E, int k, int renorm, float scale)
{
    __shared__ __attribute__((aligned(16))) float ds_lds[kThreads / LANES][LANES * 4 * Q];
    const int r = threadIdx.x % LANES;
    float* const ds_row = ds_lds[threadIdx.x / LANES];
    const int64_t t = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    const bool live = t < n_tokens;               // (a row of lanes without a token does the last one's, unstored)
    const int64_t tr = live ? t : n_tokens - 1;
    const T* const row = logits + tr * E;
    // (loads and scores without branches: behind one each of them waits for the last, which takes
    // a wave per token, 32768 x 384, from 19.7 to 21.6 us)
    int id = ids[tr * k + min(r, k - 1)];
    id = r < k && (uint32_t)id < (uint32_t)E ? id : -1;
    float dw = dweights[tr * k + min(r, k - 1)];
    dw = id >= 0 ? dw : 0.0f;
    const float lj = load_logit(row + max(id, 0));
#pragma unroll
    for (int q = 0; q < Q; ++q)
        *reinterpret_cast<f32x4*>(ds_row + (q * LANES + r) * 4) = f32x4{};
    float p[Q][4];
    RowNorm n{0.0f, 1.0f};
    Sigmoid own{0.0f, 0.0f};
    if constexpr (SIGMOID) {                      // its gradient is of the chosen alone
        own = sigmoid_f32(lj);
    } else {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int e = (q * LANES + r) * 4;
            if (VEC) {
                const f32x4 v = load_logit4(row + (e < E ? e : 0));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    p[q][j] = e < E ? v[j] : -__builtin_inff();
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float v = load_logit(row + min(e + j, E - 1));
                    p[q][j] = e + j < E ? v : -__builtin_inff();
                }
            }
        }
        float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top = fmaxf(top, p[q][j]);
        n.m = norm_top(lanes_max<LANES>(order_key(top)));
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sum += p[q][j] = exp_f32(p[q][j] - n.m);
        n.inv = norm_inv(lanes_sum<LANES>(sum));
    }
    const uint32_t sbits = __float_as_uint(SIGMOID ? own.s : softmax_of(lj, n));
    const float sj = __uint_as_float(id < 0 ? 0u : sbits);
    float ds = scale * dw;
    if (renorm) {
        const float D = lanes_sum<LANES>(sj) + 1e-20f;
        ds = scale * ((dw - lanes_sum<LANES>(dw * sj) / D) / D);
    }
    wave_lds_order();                             // the zeros are other lanes'
    if (id >= 0)
        ds_row[id] = SIGMOID ? ds * own.ds : ds;
    else
        ds = 0.0f;
    float dot = 0.0f;
    if constexpr (!SIGMOID) {
        dot = lanes_sum<LANES>(ds * sj);
        // a row without a choice may hold anything, NaN too, and has no gradient
        const uint64_t chosen = __ballot(id >= 0);
        const bool none = (LANES == 16 ? chosen >> (threadIdx.x & 48) & 0xFFFF : chosen) == 0;
        if (__ballot(none) && none) {
            n.inv = 0.0f;
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    p[q][j] = 0.0f;
        }
    }
    wave_lds_order();                             // (one wave writes and reads the row)
    T* const out = dlogits + tr * E;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = (q * LANES + r) * 4;
        const f32x4 d = *reinterpret_cast<const f32x4*>(ds_row + e);
        f32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = SIGMOID ? d[j] : p[q][j] * n.inv * (d[j] - dot);
        if (VEC) {
            if (live && e < E)
                store_logit4(out + e, v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (live && e + j < E)
                    store_logit(out + e + j, v[j]);
        }
    }
}

template <typename T>
static const void* route_kernel_for(int vpl, bool vec)
{
    switch (vpl) {
    case 1: return (const void*)route_kernel<1, false, T>;
    case 2: return (const void*)route_kernel<2, false, T>;
    case 4: return vec ? (const void*)route_kernel<4, true, T> : (const void*)route_kernel<4, false, T>;
    case 8: return vec ? (const void*)route_kernel<8, true, T> : (const void*)route_kernel<8, false, T>;
    case 16: return vec ? (const void*)route_kernel<16, true, T> : (const void*)route_kernel<16, false, T>;
    default: return (const void*)route_kernel<kMaxRouteV, false, T>;
    }
}
template <typename T>
static const void* route_quad_kernel_for(int vpl, bool vec)
{
    switch (vpl) {
    case 4: return vec ? (const void*)route_quad_kernel<4, true, T> : (const void*)route_quad_kernel<4, false, T>;
    case 8: return vec ? (const void*)route_quad_kernel<8, true, T> : (const void*)route_quad_kernel<8, false, T>;
    default: return vec ? (const void*)route_quad_kernel<16, true, T> : (const void*)route_quad_kernel<16, false, T>;
    }
}

template <bool VEC, bool SIGMOID, typename T>
static const void* route_backward_of(int lanes, int q)
{
    if (lanes == 16)
        return q == 1   ? (const void*)route_backward_kernel<16, 1, VEC, SIGMOID, T>
               : q == 2 ? (const void*)route_backward_kernel<16, 2, VEC, SIGMOID, T>
                        : (const void*)route_backward_kernel<16, 4, VEC, SIGMOID, T>;
    return q == 1   ? (const void*)route_backward_kernel<64, 1, VEC, SIGMOID, T>
           : q == 2 ? (const void*)route_backward_kernel<64, 2, VEC, SIGMOID, T>
                    : (const void*)route_backward_kernel<64, 4, VEC, SIGMOID, T>;
}
template <typename T>
static const void* route_backward_for(int lanes, int q, bool vec, bool sigmoid)
{
    if (sigmoid)
        return vec ? route_backward_of<true, true, T>(lanes, q) : route_backward_of<false, true, T>(lanes, q);
    return vec ? route_backward_of<true, false, T>(lanes, q) : route_backward_of<false, false, T>(lanes, q);
}

// Workgroups of the router at most with a wave per token: the 8 a CU holds at a time; they
// take tokens in turn.
constexpr int64_t kRouteGroups = 2048;

hipError_t launch_route(const void* logits, bool f32, const float* bias, const uint8_t* row_mask, int32_t* ids,
                        float* weights, int64_t T, int32_t E, int32_t n_group, int32_t topk_group,
                        int32_t group_best, int32_t k, bool sigmoid, bool renorm, float scale, hipStream_t stream)
{
    int gs = E / n_group, l_log = 0, vpl = 4;
    while (16 * vpl < E)
        vpl *= 2;
    // four tokens per wave if a row of 16 lanes holds the experts, and whole lanes a group
    const int per_group = gs / vpl;               // lanes
    const bool groups_fit = topk_group == n_group || (gs % vpl == 0 && per_group * n_group == 16 &&
                                                      (per_group & (per_group - 1)) == 0);
    const bool quad = vpl <= 16 && k <= 8 && groups_fit;
    const int tokens = kThreads / 64 * (quad ? 4 : 1);     // of a workgroup at a time
    if (quad) {
        while (2 << l_log <= per_group)
            ++l_log;
    } else {
        while (2 * n_group << l_log <= 64)
            ++l_log;
        const int need = (gs + (1 << l_log) - 1) >> l_log;     // experts per lane
        vpl = 1;
        while (vpl < need)
            vpl *= 2;
        if (vpl > kMaxRouteV)
            return hipErrorInvalidValue;
    }
    const int64_t need_groups = (T + tokens - 1) / tokens;
    const int64_t grid = quad || need_groups < kRouteGroups ? need_groups : kRouteGroups;
    if (grid > 0x7FFFFFFF)
        return hipErrorInvalidValue;
    int64_t t = T;
    int e = E, ng = n_group, tg = topk_group, gb = group_best, kk = k, sg = sigmoid, rn = renorm;
    float sc = scale;
    void* args[] = {(void*)&logits, (void*)&bias, (void*)&row_mask, (void*)&ids, (void*)&weights, (void*)&t, (void*)&e,
                    (void*)&ng, (void*)&gs, (void*)&tg, (void*)&gb, (void*)&kk, (void*)&sg, (void*)&rn, (void*)&sc,
                    (void*)&l_log};
    const bool vec = quad ? E % 4 == 0 : gs % 4 == 0;      // rows (and a lane's part of them) are aligned
    const void* kernel;
    if (quad)
        kernel = f32 ? route_quad_kernel_for<float>(vpl, vec) : route_quad_kernel_for<uint16_t>(vpl, vec);
    else
        kernel = f32 ? route_kernel_for<float>(vpl, vec) : route_kernel_for<uint16_t>(vpl, vec);
    return launch_kernel(kernel, dim3((unsigned)grid), dim3(kThreads), args, stream);
}

hipError_t launch_route_backward(const void* logits, bool f32, const int32_t* ids, const float* dweights,
                                 void* dlogits, int64_t T, int32_t E, int32_t k, bool sigmoid, bool renorm,
                                 float scale, hipStream_t stream)
{
    // a row of 16 lanes per token where it holds the choices and 16 experts a lane: 32768 x 60,
    // BF16: 4.5 us, a wave per token 11.7; 16384 x 256, FP32: 7.9 and 8.6
    const int lanes = E <= 256 && k <= 16 ? 16 : 64;
    int q = 1;
    while (4 * lanes * q < E)
        q *= 2;
    const int per = kThreads / lanes;             // tokens of a workgroup
    const int64_t grid = (T + per - 1) / per;
    int64_t t = T;
    int e = E, kk = k, rn = renorm;
    float sc = scale;
    void* args[] = {(void*)&logits, (void*)&ids, (void*)&dweights, (void*)&dlogits, (void*)&t, (void*)&e,
                    (void*)&kk, (void*)&rn, (void*)&sc};
    const bool vec = E % 4 == 0;
    const void* kernel = f32 ? route_backward_for<float>(lanes, q, vec, sigmoid)
                             : route_backward_for<uint16_t>(lanes, q, vec, sigmoid);
    return launch_kernel(kernel, dim3((unsigned)grid), dim3(kThreads), args, stream);
}

}  // namespace mxfp4
