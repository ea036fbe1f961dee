// Stores of rows that the same kernel does not read again, with the non-temporal
// hint: they leave L2's retained lines to what is read several times, and the
// write stream no longer waits for lines to be evicted.
#pragma once
#include "rng.h"

namespace mok {

typedef uint32_t u32x4_nt_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_nt_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void stream16(void *base, int64_t i, uint4 v) {   // the i-th 16 bytes
    const u32x4_nt_t w = {v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(w, static_cast<u32x4_nt_t *>(base) + i);
}
__device__ __forceinline__ void stream8(void *base, int64_t i, uint2 v) {    // the i-th 8 bytes
    const u32x2_nt_t w = {v.x, v.y};
    __builtin_nontemporal_store(w, static_cast<u32x2_nt_t *>(base) + i);
}
// 8 elements of the residual stream's types, rounded (store8) or as they were loaded.
template <Elem E>
__device__ __forceinline__ void stream8_elems(void *base, int64_t c, const float (&f)[8]) {
    if constexpr (E == kBf16) {
        stream16(base, c, pack8_bf16(f));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            stream16(base, 2 * c + i, make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                                 __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3])));
    }
}
template <Elem E>
__device__ __forceinline__ void stream8_raw(void *base, int64_t c, const Raw8<E> &r) {
    if constexpr (E == kBf16) {
        stream16(base, c, r.v);
    } else {
        stream16(base, 2 * c, r.lo);
        stream16(base, 2 * c + 1, r.hi);
    }
}

}  // namespace mok
