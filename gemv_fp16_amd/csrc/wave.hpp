// Reductions over the 64 lanes of a wave, through DPP moves (no LDS).
#pragma once
#include "common.hpp"

namespace gf {

// One DPP move of 32 bits; lanes without a source keep `old`.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_move(int old, int v)
{
    return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xF, false);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_move(float old, float v)
{
    return __builtin_bit_cast(float, dpp_move<CTRL, ROWS>(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v)));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_move(double old, double v)
{
    typedef int int2v __attribute__((ext_vector_type(2)));
    const int2v o = __builtin_bit_cast(int2v, old), x = __builtin_bit_cast(int2v, v);
    int2v r;
    r.x = dpp_move<CTRL, ROWS>(o.x, x.x);
    r.y = dpp_move<CTRL, ROWS>(o.y, x.y);
    return __builtin_bit_cast(double, r);
}

__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

__device__ __forceinline__ double lane_value(double v, int lane)
{
    typedef int int2v __attribute__((ext_vector_type(2)));
    int2v x = __builtin_bit_cast(int2v, v);
    x.x = __builtin_amdgcn_readlane(x.x, lane);
    x.y = __builtin_amdgcn_readlane(x.y, lane);
    return __builtin_bit_cast(double, x);
}

// op over all lanes (every lane must be active): within the rows of 16 by quad
// permutes and mirrors, then row 0 into 1 and 2 into 3, then both into lane 63.
// `id` is op's identity.  Wave-uniform, always the same order.
template <class T, class Op>
__device__ __forceinline__ T wave_reduce(T v, T id, Op op)
{
    v = op(v, dpp_move<0xB1, 0xF>(id, v));     // lanes 1 0 3 2
    v = op(v, dpp_move<0x4E, 0xF>(id, v));     // lanes 2 3 0 1
    v = op(v, dpp_move<0x141, 0xF>(id, v));    // mirrored within 8
    v = op(v, dpp_move<0x140, 0xF>(id, v));    // mirrored within 16
    v = op(v, dpp_move<0x142, 0xA>(id, v));    // lane 15 of rows 0, 2 into rows 1, 3
    v = op(v, dpp_move<0x143, 0xC>(id, v));    // lane 31 into rows 2, 3
    return lane_value(v, kWave - 1);
}

// The same within each row of 16 lanes, where every lane gets its row's result.
template <class T, class Op>
__device__ __forceinline__ T row_reduce(T v, T id, Op op)
{
    v = op(v, dpp_move<0xB1, 0xF>(id, v));
    v = op(v, dpp_move<0x4E, 0xF>(id, v));
    v = op(v, dpp_move<0x141, 0xF>(id, v));
    return op(v, dpp_move<0x140, 0xF>(id, v));
}

// The largest over the lanes l, l + MT, l + 2 MT .. of each l, in all of them.
template <int MT>
__device__ __forceinline__ float rows_max(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    auto larger = [](auto p) {
        return __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
    };
    v = larger(__builtin_amdgcn_permlane32_swap(b, b, false, false));
    if constexpr (MT == 16) {
        const uint32_t c = __builtin_bit_cast(uint32_t, v);
        v = larger(__builtin_amdgcn_permlane16_swap(c, c, false, false));
    }
    return v;
}

// A NaN loses to any number.
__device__ __forceinline__ float wave_max(float v)
{
    return wave_reduce(v, -__builtin_inff(), [](float a, float b) { return __builtin_fmaxf(a, b); });
}

template <class T>
__device__ __forceinline__ T wave_sum(T v)
{
    return wave_reduce(v, T(0), [](T a, T b) { return a + b; });
}

// Inclusive sums over the lanes (every lane active): within the rows of 16, then rows
// 0, 2 into 1, 3, and the first two into the others.
__device__ __forceinline__ int wave_scan(int v)
{
    v += dpp_move<0x111, 0xF>(0, v);           // from the lane 1 below, 2, 4, 8
    v += dpp_move<0x112, 0xF>(0, v);
    v += dpp_move<0x114, 0xF>(0, v);
    v += dpp_move<0x118, 0xF>(0, v);
    v += dpp_move<0x142, 0xA>(0, v);
    v += dpp_move<0x143, 0xC>(0, v);
    return v;
}

}  // namespace gf
