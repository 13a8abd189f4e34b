// Sums, running sums and maxima over the 64 lanes of a wave by data-parallel row shifts: no LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace w4a16 {

template <int kCtrl, int kRows, class T>
__device__ __forceinline__ T lane_shift(T v, T none) {             // lanes without a source take `none`
    if constexpr (sizeof(T) == 8) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v), n = __builtin_bit_cast(uint64_t, none);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)n, (int)(uint32_t)b, kCtrl, kRows, 0xF, false);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(n >> 32), (int)(b >> 32), kCtrl, kRows, 0xF, false);
        return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v), kCtrl, kRows, 0xF, false));
    }
}
template <class T>
__device__ __forceinline__ T from_lane(T v, int lane) {            // lane: the same in all lanes
    if constexpr (sizeof(T) == 8) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane), hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane);
        return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
    }
}

// op over lanes 0 .. own; `none` changes nothing under it
template <class T, class Op>
__device__ __forceinline__ T wave_scan(T v, T none, Op op) {
    v = op(v, lane_shift<0x111, 0xF>(v, none));      // row_shr 1, 2, 4, 8
    v = op(v, lane_shift<0x112, 0xF>(v, none));
    v = op(v, lane_shift<0x114, 0xF>(v, none));
    v = op(v, lane_shift<0x118, 0xF>(v, none));
    v = op(v, lane_shift<0x142, 0xA>(v, none));      // lane 15 of a row to the next row
    return op(v, lane_shift<0x143, 0xC>(v, none));   // lane 31 to the upper half
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
    return from_lane(wave_scan(v, T(0), [](T a, T b) { return a + b; }), 63);
}
// the sum over the lower lanes, and over all
template <class T>
__device__ __forceinline__ T wave_before(T v, T* all) {
    const T sum = wave_scan(v, T(0), [](T a, T b) { return a + b; });
    *all = from_lane(sum, 63);
    return lane_shift<0x138, 0xF>(sum, T(0));        // one lane up
}
__device__ __forceinline__ float wave_max(float v) {
    return from_lane(wave_scan(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); }), 63);
}
__device__ __forceinline__ double wave_max(double v) {
    return from_lane(wave_scan(v, (double)-INFINITY, [](double a, double b) { return fmax(a, b); }), 63);
}

}  // namespace w4a16
