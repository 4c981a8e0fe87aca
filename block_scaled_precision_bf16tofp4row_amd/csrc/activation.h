// activation.h -- activations and their derivatives in FP32, and eight FP32 values to and from
// BF16 and to E4M3 under the FP32 scale of their 1x128 block.
//
// With e = exp(-x) or exp(-x^2 / 2) from the hardware's 2^x (2^-23, and the argument E's own
// roundings, 1 to 6 times E 2^-24) and the hardware's reciprocal (2^-23); tests/act_bounds.py has
// the bounds that follow, and the header states them:
//   relu       max(x, 0); derivative 1 where x > 0, else 0
//   silu       x s, s = 1 / (1 + exp(-x)); derivative s (1 + x (1 - s))
//   gelu       x P(x), P the normal distribution; derivative P + x exp(-x^2 / 2) / sqrt(2 pi).
//              P(-z) = t Q(t) exp(-z^2 / 2) for z >= 0, t = 1 / (1 + 0.28 z), Q of degree 8 (a
//              least-squares fit of its relative error, reweighted to be even: 1.8e-7; 5.3e-7 to 6.5e-7
//              evaluated in FP32 with z up to 4), and P(z) = 1 - P(-z): one exponential for value and
//              derivative, and small values on the left keep their precision, which 1 + erf
//              there would not
//   gelu_tanh  x s, s = 1 / (1 + exp(-2 c (x + 0.044715 x^3))), c = sqrt(2 / pi), which is the
//              usual form with the hyperbolic tangent
// A NaN gives NaN in both.  Where a formula has infinity times zero it gives NaN too: silu and
// gelu at -inf, their derivatives at both infinities, and gelu_tanh at -inf (its derivative is 1
// and 0 there).
#pragma once

#include <type_traits>

#include "lanes.h"

namespace mxfp4 {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// f and, if kSlope, f' of x.  ACT: one of Act.
template <int ACT, bool kSlope>
__device__ __forceinline__ void activate(float x, float& f, float& slope)
{
    if constexpr (ACT == kActNone) {
        f = x;
        slope = 1.0f;
    } else if constexpr (ACT == kActRelu) {
        f = x < 0.0f ? 0.0f : x;
        slope = x <= 0.0f ? 0.0f : x > 0.0f ? 1.0f : x;
    } else if constexpr (ACT == kActSilu) {
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-x));
        f = x * s;
        if constexpr (kSlope)
            slope = s * __builtin_fmaf(x, 1.0f - s, 1.0f);
    } else if constexpr (ACT == kActGelu) {
        const float z = fabsf(x), t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.28f, z, 1.0f));
        const float e = __expf(-0.5f * x * x);
        float q = 0.024720078334212303f;
        q = __builtin_fmaf(q, t, -0.09359350055456161f);
        q = __builtin_fmaf(q, t, 0.09242866188287735f);
        q = __builtin_fmaf(q, t, -0.006449582055211067f);
        q = __builtin_fmaf(q, t, 0.07277517020702362f);
        q = __builtin_fmaf(q, t, 0.0836307555437088f);
        q = __builtin_fmaf(q, t, 0.10308466851711273f);
        q = __builtin_fmaf(q, t, 0.11169980466365814f);
        q = __builtin_fmaf(q, t, 0.11170385777950287f);
        q *= t * e;
        const float p = x < 0.0f ? q : 1.0f - q;
        f = x * p;
        if constexpr (kSlope)
            slope = __builtin_fmaf(x, 0.3989422804014327f * e, p);
    } else {
        constexpr float kC = 1.5957691216057308f;                        // 2 sqrt(2 / pi)
        const float y = fabsf(x) > 30.0f ? copysignf(30.0f, x) : x;      // (x^2 0 past it, not inf 0)
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-kC * y * __builtin_fmaf(0.044715f * y, y, 1.0f)));
        f = x * s;
        if constexpr (kSlope)
            slope = s * __builtin_fmaf(y * (1.0f - s), kC * __builtin_fmaf(0.134145f * y, y, 1.0f), 1.0f);
    }
}

// f (in place of x) and, if kSlope, f' of eight values; act is the same in all lanes.
template <bool kSlope>
__device__ __forceinline__ void activate8(int act, float (&x)[8], float (&slope)[8])
{
    auto all = [&](auto a) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            activate<decltype(a)::value, kSlope>(x[i], x[i], slope[i]);
    };
    switch (act) {
    case kActRelu: all(std::integral_constant<int, kActRelu>{}); break;
    case kActSilu: all(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: all(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: all(std::integral_constant<int, kActGeluTanh>{}); break;
    default: all(std::integral_constant<int, kActNone>{}); break;
    }
}

__device__ __forceinline__ u32x4 to_bf16(const float (&v)[8])
{
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2 p = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
        r[i] = __builtin_bit_cast(uint32_t, p);
    }
    return r;
}
__device__ __forceinline__ void from_bf16(u32x4 r, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(r[i] << 16);
        v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
}

// Eight values of a 1x128 block that the 16 lanes of a row hold -> E4M3 bytes and the block's
// scale: with a = max(amax, 2^-100), scale = a / 448 and byte = E4M3(x * (448 / a)).
__device__ __forceinline__ u32x2 to_fp8(const float (&v)[8], float& scale)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const float a = fmaxf(__uint_as_float(row_max(m)), 0x1p-100f);
    const float mul = 448.0f / a;
    scale = a / 448.0f;
    u32x2 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * mul, v[4 * i + 1] * mul, 0, false);
        r[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * mul, v[4 * i + 3] * mul, w, true);
    }
    return r;
}

}  // namespace mxfp4
