// Folds across the lanes of a wave.
#pragma once

#include <hip/hip_runtime.h>

namespace ssm {

// f folded over the 64 lanes, in every lane, in a fixed order: exchanges inside
// each row of 16 lanes by DPP patterns, between the rows by permlane swaps (no
// LDS round trips).
template <int CTRL> __device__ __forceinline__ float dpp_get(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
// L < 64: over each aligned run of L lanes (8, 16, 32).
template <int L = 64, typename F> __device__ __forceinline__ float wave_fold(float v, F f) {
    static_assert(L == 8 || L == 16 || L == 32 || L == 64, "runs of lanes");
    v = f(v, dpp_get<0xB1>(v));       // quad_perm 1,0,3,2
    v = f(v, dpp_get<0x4E>(v));       // quad_perm 2,3,0,1
    v = f(v, dpp_get<0x141>(v));      // row_half_mirror: the other quad of 8 lanes
    if constexpr (L >= 16) v = f(v, dpp_get<0x140>(v));   // row_mirror: the other half of 16 lanes
    if constexpr (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    if constexpr (L == 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}
struct AddOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

}  // namespace ssm
