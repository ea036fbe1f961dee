// Sums across the lanes of a wave on the vector unit alone (DPP and the lane
// swaps of gfx950). __shfl_xor goes through the LDS pipe, about 100 cycles a
// dependent step: the six steps of a wave sum then cost more than the few
// loads they follow. Both partners of a step add the same two values, so every
// lane of a group ends with the same bits.
#pragma once
#include "common.h"

namespace mok {

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {   // x + (x of the lane that CTRL names)
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E;     // quad_perm [1,0,3,2], [2,3,0,1]
constexpr int kDppRor4 = 0x124, kDppRor8 = 0x128;   // rotations inside a row of 16 lanes
constexpr int kDppHalfMirror = 0x141;               // lane i of 8 takes lane 7 - i

// Lanes 16 apart: the swap leaves rows (0, 0, 2, 2) in one register and (1, 1, 3, 3) in the other.
__device__ __forceinline__ float add_xor16(float x) {
    const uint32_t b = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Lanes 32 apart: (low, low) and (high, high).
__device__ __forceinline__ float add_xor32(float x) {
    const uint32_t b = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over the lanes that differ in the bits FROM .. 32 of their index (FROM = 4 or 8).
template <int FROM>
__device__ __forceinline__ float sum_lanes(float x) {
    static_assert(FROM == 4 || FROM == 8, "4 or 8 lanes stay apart");
    x = dpp_add<kDppRor8>(x);
    if constexpr (FROM == 4) x = dpp_add<kDppRor4>(x);   // equal 8 apart by now, so a rotation by 4 is the exchange
    return add_xor32(add_xor16(x));
}

// Sum over groups of `lanes` neighbouring lanes (8, 16, 32 or 64, the same for the whole wave).
__device__ __forceinline__ float sum_group(float x, int lanes) {
    x = dpp_add<kDppXor2>(dpp_add<kDppXor1>(x));
    x = dpp_add<kDppHalfMirror>(x);                  // equal within fours by now
    if (lanes >= 16) x = dpp_add<kDppRor8>(x);
    if (lanes >= 32) x = add_xor16(x);
    if (lanes >= 64) x = add_xor32(x);
    return x;
}

__device__ __forceinline__ float sum_wave(float x) { return sum_group(x, 64); }

}  // namespace mok
