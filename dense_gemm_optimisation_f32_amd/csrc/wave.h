// wave.h -- reductions and sums over the 64 lanes of a wave by DPP moves (no LDS
// traffic): within rows of 16 lanes, then across rows; the whole result arrives in
// lane 63.  All lanes take part in each.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mi355gemm {
namespace {

template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned dpp(unsigned old, unsigned v)
{
    return (unsigned)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float old, float v)
{
    return __builtin_bit_cast(float, dpp<CTRL, ROWS>(__builtin_bit_cast(unsigned, old), __builtin_bit_cast(unsigned, v)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double old, double v)
{
    const uint64_t o = __builtin_bit_cast(uint64_t, old), b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = dpp<CTRL, ROWS>((unsigned)o, (unsigned)b);
    const uint64_t hi = dpp<CTRL, ROWS>((unsigned)(o >> 32), (unsigned)(b >> 32));
    return __builtin_bit_cast(double, (hi << 32) | lo);
}
__device__ __forceinline__ unsigned lane_value(unsigned v, int lane)
{
    return (unsigned)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __builtin_bit_cast(float, lane_value(__builtin_bit_cast(unsigned, v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = lane_value((unsigned)b, lane), hi = lane_value((unsigned)(b >> 32), lane);
    return __builtin_bit_cast(double, (hi << 32) | lo);
}
// op(all lanes), `none` being op's neutral value; the same in every lane.
template <class T, class Op>
__device__ __forceinline__ T wave_reduce(T v, T none, Op op)
{
    v = op(v, dpp<0x111, 0xF>(none, v));   // one lane down the row, then 2, 4, 8
    v = op(v, dpp<0x112, 0xF>(none, v));
    v = op(v, dpp<0x114, 0xF>(none, v));
    v = op(v, dpp<0x118, 0xF>(none, v));
    v = op(v, dpp<0x142, 0xA>(none, v));   // each odd row takes the row before it
    v = op(v, dpp<0x143, 0xC>(none, v));   // the upper half takes the lower
    return lane_value(v, 63);
}
__device__ __forceinline__ unsigned wave_max(unsigned v)
{
    return wave_reduce(v, 0u, [](unsigned a, unsigned b) { return a > b ? a : b; });
}
__device__ __forceinline__ float wave_max(float v)   // NaN only if every lane is
{
    return wave_reduce(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}
template <class T>
__device__ __forceinline__ T wave_sum(T v)
{
    return wave_reduce(v, T(0), [](T a, T b) { return a + b; });
}
// Sums over the lanes up to and including one's own.
__device__ __forceinline__ int wave_scan(int v)
{
    auto add = [&](unsigned o) { v += (int)o; };
    add(dpp<0x111, 0xF>(0u, (unsigned)v));
    add(dpp<0x112, 0xF>(0u, (unsigned)v));
    add(dpp<0x114, 0xF>(0u, (unsigned)v));
    add(dpp<0x118, 0xF>(0u, (unsigned)v));
    add(dpp<0x142, 0xA>(0u, (unsigned)v));
    add(dpp<0x143, 0xC>(0u, (unsigned)v));
    return v;
}

}  // namespace
}  // namespace mi355gemm
