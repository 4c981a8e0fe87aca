// lanes.h -- sums and maxima over a wave and over its rows of 16 lanes, by DPP, and the order
// of a wave's own LDS accesses.
#pragma once

#include "strips.h"

namespace mxfp4 {

// (two quad permutations, the mirrors of 8 and 16 lanes, then lane 15 of a row to the next
// and lane 31 to the upper half: lane 63 has everything.)
constexpr int kRowMirror = 0x140, kRowHalfMirror = 0x141, kRowBcast15 = 0x142, kRowBcast31 = 0x143;

// What lanes of this wave wrote to LDS before it, every lane of the wave reads after it.  No
// instruction: a wave's LDS accesses are carried out in order, but without this the compiler
// need not keep accesses of different lanes to one place in it.
__device__ __forceinline__ void wave_lds_order()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Lanes that a broadcast does not reach take 0, the identity of both reductions below (keys
// and sums), so that the compiler folds the move into the operation.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_rows(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max(v, dpp<kQuadSwap1>(v));
    v = max(v, dpp<kQuadSwap2>(v));
    v = max(v, dpp<kRowHalfMirror>(v));
    v = max(v, dpp<kRowMirror>(v));
    v = max(v, dpp_rows<kRowBcast15, 0xA>(v));
    v = max(v, dpp_rows<kRowBcast31, 0xC>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float f)
{
    auto add = [&](uint32_t o) { f += __uint_as_float(o); };
    add(dpp<kQuadSwap1>(__float_as_uint(f)));
    add(dpp<kQuadSwap2>(__float_as_uint(f)));
    add(dpp<kRowHalfMirror>(__float_as_uint(f)));
    add(dpp<kRowMirror>(__float_as_uint(f)));
    add(dpp_rows<kRowBcast15, 0xA>(__float_as_uint(f)));
    add(dpp_rows<kRowBcast31, 0xC>(__float_as_uint(f)));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), 63));
}
// The sum over lanes 0 .. own: shifts by 1, 2, 4 and 8 within the rows of 16, then as above.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v)
{
    v += dpp_rows<0x111, 0xF>(v);
    v += dpp_rows<0x112, 0xF>(v);
    v += dpp_rows<0x114, 0xF>(v);
    v += dpp_rows<0x118, 0xF>(v);
    v += dpp_rows<kRowBcast15, 0xA>(v);
    return v + dpp_rows<kRowBcast31, 0xC>(v);
}
// Over the 16 lanes of a row, the result in all of them.
__device__ __forceinline__ float row_sum(float f)
{
    f += __uint_as_float(dpp<kQuadSwap1>(__float_as_uint(f)));
    f += __uint_as_float(dpp<kQuadSwap2>(__float_as_uint(f)));
    f += __uint_as_float(dpp<kRowHalfMirror>(__float_as_uint(f)));
    return f + __uint_as_float(dpp<kRowMirror>(__float_as_uint(f)));
}
__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    v = max(v, dpp<kQuadSwap1>(v));
    v = max(v, dpp<kQuadSwap2>(v));
    v = max(v, dpp<kRowHalfMirror>(v));
    return max(v, dpp<kRowMirror>(v));
}
}  // namespace mxfp4
