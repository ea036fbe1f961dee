// Counter-based random words for dropout: Philox4x32 with 10 rounds (Salmon,
// Moraes, Dror, Shaw, "Parallel Random Numbers: As Easy as 1, 2, 3", SC 2011).
// A block of four words is a pure function of a 64-bit key and a 64-bit
// counter, so a mask is recomputed wherever it is needed and never stored:
//   element i is word i % 4 of the block with counter offset + i / 4, key seed
//   kept when that word >= floor(p * 2^32); a kept value is scaled by 1 / (1 - p)
// seed and offset come from device memory, so that replays of a captured
// graph draw fresh masks once the caller has advanced them.
#pragma once
#include "common.h"

namespace mok {

// What a kernel needs of a dropout: the device state and the host-made constants.
struct DropArgs {
    const uint64_t *rng;   // {seed, offset}; null: keep everything, unscaled
    uint32_t threshold;    // floor(p * 2^32)
    float scale;           // 1 / (1 - p)
};

inline DropArgs drop_args(float p, const uint64_t *rng) {
    if (p == 0.0f) return DropArgs{nullptr, 0u, 1.0f};
    return DropArgs{rng, (uint32_t)((double)p * 4294967296.0), (float)(1.0 / (1.0 - (double)p))};
}

struct DropState {
    uint32_t k0, k1;
    uint64_t offset;
};
__device__ __forceinline__ DropState drop_state(const uint64_t *rng) {
    const uint64_t seed = rng[0];
    return DropState{(uint32_t)seed, (uint32_t)(seed >> 32), rng[1]};
}

__device__ __forceinline__ uint4 philox4x32_10(uint64_t counter, uint32_t k0, uint32_t k1) {
    uint32_t x0 = (uint32_t)counter, x1 = (uint32_t)(counter >> 32), x2 = 0, x3 = 0;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)x0 * 0xD2511F53u, p1 = (uint64_t)x2 * 0xCD9E8D57u;
        const uint32_t y0 = (uint32_t)(p1 >> 32) ^ x1 ^ k0, y2 = (uint32_t)(p0 >> 32) ^ x3 ^ k1;
        x1 = (uint32_t)p1;
        x3 = (uint32_t)p0;
        x0 = y0;
        x2 = y2;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
}

// The words of elements [8c, 8c + 8).
struct Words8 {
    uint32_t w[8];
};
__device__ __forceinline__ Words8 drop_words8(const DropState &st, int64_t c) {
    const uint64_t ctr = st.offset + 2u * (uint64_t)c;
    const uint4 a = philox4x32_10(ctr, st.k0, st.k1), b = philox4x32_10(ctr + 1, st.k0, st.k1);
    return Words8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// Element kinds of the residual stream and eight of them in registers.
enum Elem { kNone = 0, kBf16 = 1, kF32 = 2 };
template <Elem E>
struct Raw8 {   // 8 elements as loaded (kNone: nothing)
};
template <>
struct Raw8<kBf16> {
    uint4 v;
};
template <>
struct Raw8<kF32> {
    uint4 lo, hi;
};
template <Elem E>
__device__ __forceinline__ Raw8<E> load8(const void *base, int64_t c) {
    if constexpr (E == kBf16) return Raw8<E>{static_cast<const uint4 *>(base)[c]};
    if constexpr (E == kF32)
        return Raw8<E>{static_cast<const uint4 *>(base)[2 * c], static_cast<const uint4 *>(base)[2 * c + 1]};
    return Raw8<E>{};
}
template <Elem E>
__device__ __forceinline__ void unpack8(const Raw8<E> &r, float (&f)[8]) {
    if constexpr (E == kBf16) {
        const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else if constexpr (E == kF32) {
        const uint32_t w[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.0f;
    }
}
__device__ __forceinline__ uint4 pack8_bf16(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
template <Elem E>
__device__ __forceinline__ void store8(void *base, int64_t c, const float (&f)[8]) {
    if constexpr (E == kBf16) {
        static_cast<uint4 *>(base)[c] = pack8_bf16(f);
    } else if constexpr (E == kF32) {
        uint4 *p = static_cast<uint4 *>(base) + 2 * c;
        p[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        p[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    }
}

// base + dropped x: a kept value is one fused multiply-add, a dropped one
// leaves base as it is (also where x holds an infinity or a NaN).
__device__ __forceinline__ float drop_add(float x, uint32_t word, const DropArgs &d, float base) {
    return word >= d.threshold ? __builtin_fmaf(x, d.scale, base) : base;
}

}  // namespace mok
