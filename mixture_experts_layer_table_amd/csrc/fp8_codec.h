// Blocks of 128 values with one fp32 scale and E4M3FN elements: scale = m / 448
// and element = E4M3FN(v * (448 / m)) with m = max(largest magnitude, 2^-52).
// The floor keeps the product of two scales a normal fp32 number (2^-122 at
// least); a block whose largest magnitude lies below it still rounds its values
// relative to E4M3's smallest normal, 2^-6, so nothing is lost down to 2^-67.
// A block that holds a NaN or an infinity has no such scale: its elements become
// NaN throughout and its scale 1, so that every product with it shows it.
#pragma once
#include "mx_codec.h"

namespace mok {

constexpr int kBlk = 128;

struct BlkScale {
    float scale, mul;
    uint32_t nan;   // in place of four codes where it is not 0
};
// amax_bits: bits of the block's largest |fp32| (a NaN's lie above infinity's).
__device__ __forceinline__ BlkScale blk_scale(uint32_t amax_bits) {
    const bool bad = amax_bits >= 0x7F800000u;
    const float m = bad ? 448.0f : fmaxf(__uint_as_float(amax_bits), 0x1p-52f);
    return BlkScale{m / 448.0f, 448.0f / m, bad ? 0x7F7F7F7Fu : 0u};
}
constexpr float kLeastScale = 0x1p-52f / 448.0f;   // of a block of zeros

__device__ __forceinline__ uint32_t blk_codes4(const BlkScale &b, float v0, float v1, float v2, float v3) {
    const uint32_t q = e4m3x2_scaled(v0 * b.mul, v1 * b.mul) | (e4m3x2_scaled(v2 * b.mul, v3 * b.mul) << 16);
    return b.nan ? b.nan : q;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
    return m;
}

// Largest of the 16 lanes of a row of lanes; every lane of the 16 takes part.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t max16(uint32_t x) {
    x = dpp_max<0xB1>(x);          // quad_perm [1,0,3,2]
    x = dpp_max<0x4E>(x);          // quad_perm [2,3,0,1]
    x = dpp_max<0x124>(x);         // rotations by 4 and 8 inside the 16
    return dpp_max<0x128>(x);
}

// The same of 8 neighbouring lanes.
__device__ __forceinline__ uint32_t max8(uint32_t x) {
    x = dpp_max<0xB1>(x);
    x = dpp_max<0x4E>(x);
    return dpp_max<0x141>(x);      // lane i of 8 takes lane 7 - i: equal within fours by now
}

}  // namespace mok
