// zsp_wave.hpp -- joining one 64-bit value per lane over a wave, for the norm
// kernels. Device code only.
//
// Four DPP steps join the lanes of each row of 16 (a lane takes its
// neighbour's, then across pairs, then mirrored in 8 and in 16 lanes), and
// the four rows are read as scalars: no LDS, no waits on it. A wave of a
// reduce with a norm joins once per 256 or 512 elements, at its very end,
// where the six LDS steps of a shuffle tree lengthened every wave's life.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace zsp {

template <int CTRL>
__device__ __forceinline__ double dpp_move(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo =
        __builtin_amdgcn_mov_dpp(int(uint32_t(u)), CTRL, 0xf, 0xf, true);
    const uint32_t hi =
        __builtin_amdgcn_mov_dpp(int(uint32_t(u >> 32)), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

__device__ __forceinline__ double read_lane(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(int(uint32_t(u)), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(int(uint32_t(u >> 32)), lane);
    return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// op over all 64 lanes (all active), in a fixed order; the same in every lane.
template <typename Op>
__device__ __forceinline__ double wave_join(double v, Op op) {
    v = op(v, dpp_move<0xB1>(v));   // quad_perm 1 0 3 2
    v = op(v, dpp_move<0x4E>(v));   // quad_perm 2 3 0 1
    v = op(v, dpp_move<0x141>(v));  // row_half_mirror
    v = op(v, dpp_move<0x140>(v));  // row_mirror
    return op(op(read_lane(v, 0), read_lane(v, 16)), op(read_lane(v, 32), read_lane(v, 48)));
}

// Joins two sums of squares, or two largest absolute values: non-negative
// numbers, or NaN with a clear sign, whose bit patterns order as integers.
struct JoinSum {
    __device__ __forceinline__ double operator()(double a, double b) const { return a + b; }
};
struct JoinMax {
    __device__ __forceinline__ double operator()(double a, double b) const {
        const uint64_t x = __builtin_bit_cast(uint64_t, a), y = __builtin_bit_cast(uint64_t, b);
        return __builtin_bit_cast(double, x > y ? x : y);
    }
};

}  // namespace zsp
