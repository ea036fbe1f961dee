// Quantization of a 32-block held by two lanes of an MFMA accumulator, for the
// epilogues of the block-scaled products.
#pragma once
#include "mx_codec.h"

namespace mok {
namespace {

// Quantize 16 fp32 values a lane holds of one 32-block (its partner lane
// l ^ 32 holds the other 16, columns g4*8 + 4*(l/32) + j of the block).
// Returns the scale byte and, in enc[g4], the 4 codes of columns
// g4*8 + 4h .. +3. Every lane of the wave must call this (cross-lane
// exchange). quantize_block16 is kept out of line: epilogues call it up to 16
// times, and inlining every copy would stop the accumulator loops from
// unrolling. A call waits for every load and store in flight, though; an
// epilogue that keeps stores in flight uses encode_block16.
struct Block16 {
    float v[16];
};
struct Enc16 {
    uint32_t enc[4];
    uint32_t scale;
};
__device__ __forceinline__ Enc16 encode_block16(const Block16 &b) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = max(amax, __float_as_uint(b.v[i]) & 0x7FFFFFFFu);
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 32));
    Enc16 r;
    r.scale = mx_scale_byte_f32(amax);
    const float sc = mx_pow2_neg((int)r.scale - 127);
    const uint32_t nan = mx_nan_f32(amax);
#pragma unroll
    for (int g4 = 0; g4 < 4; ++g4)
        r.enc[g4] = nan | e4m3x2_scaled(b.v[g4 * 4] * sc, b.v[g4 * 4 + 1] * sc) |
                    (e4m3x2_scaled(b.v[g4 * 4 + 2] * sc, b.v[g4 * 4 + 3] * sc) << 16);
    return r;
}
__device__ __attribute__((noinline)) Enc16 quantize_block16(Block16 b) { return encode_block16(b); }

}  // namespace
}  // namespace mok
