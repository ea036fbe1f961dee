// What the kernels of the products on blocks of 128 share.
#pragma once
#include "fp8_gemm.h"
#include "layer_parts.h"

namespace mok {

struct BlkArgs {
    int64_t xs_ld, ws_ld;    // entries from one block's scales to the next (X; W by rows)
    const uint8_t *x, *w;
    const float *xs, *ws;
    const int32_t *offsets;  // NULL: one product
    const void *addend;
    void *out;
    int M, N, K, E;          // output rows (of all experts together, or of one), columns, contraction
    int ld;                  // bytes from row to row, of both
    int splits, run;         // runs of the contraction, and a product by weights' K-blocks in one
    float *part;             // more than one run: fp32 partials, [splits] outputs
};

__device__ __forceinline__ int clamp_row(int v, int M) { return min(max(v, 0), M); }
__device__ __forceinline__ int uniform_i(int v) { return __builtin_amdgcn_readfirstlane(v); }

// First row of expert e (lane-wise) and its rows; E = 0: one product of all rows.
__device__ __forceinline__ int expert_rows(const BlkArgs &a, int e, int &lo) {
    lo = 0;
    if (a.E == 0) return e == 0 ? a.M : 0;
    if (e >= a.E) return 0;
    lo = clamp_row(a.offsets[e], a.M);
    return max(clamp_row(a.offsets[e + 1], a.M) - lo, 0);
}
__device__ __forceinline__ int lane_scan(int v) {   // inclusive
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if ((int)(threadIdx.x & 63) >= d) v += o;
    }
    return v;
}
// Sum over the experts of count(rows); and the expert that the i-th of them belongs to.
template <class F>
__device__ __forceinline__ int count_tiles(const BlkArgs &a, F &&count) {
    int total = 0, lo;
    for (int e0 = 0; e0 < max(a.E, 1); e0 += 64)
        total += __shfl(lane_scan(count(expert_rows(a, e0 + (int)(threadIdx.x & 63), lo))), 63);
    return uniform_i(total);
}
struct Found {
    int e, lo, n, i;   // the expert, its first row and rows, which of its tiles
};
template <class F>
__device__ __forceinline__ Found find_tile(const BlkArgs &a, int i, F &&count) {
    int before = 0;
    for (int e0 = 0; e0 < max(a.E, 1); e0 += 64) {
        int lo;
        const int n = expert_rows(a, e0 + (int)(threadIdx.x & 63), lo), c = count(n), incl = before + lane_scan(c);
        const uint64_t past = __ballot(incl > i);
        if (past) {
            const int who = __builtin_ctzll(past);
            return Found{uniform_i(e0 + who), uniform_i(__shfl(lo, who)), uniform_i(__shfl(n, who)),
                         uniform_i(i - __shfl(incl - c, who))};
        }
        before = __shfl(incl, 63);
    }
    return Found{-1, 0, 0, 0};   // i is not below the sum
}

// The product by weights for few rows (fp8_few.hip): mt tiles of 16 rows at a time (1, 2 or 4), nw tiles of 16 weight
// rows a workgroup (1 or 2).
hipError_t launch_blk_few(const BlkArgs &a, int mt, int nw, bool f32, hipStream_t st);

}  // namespace mok
