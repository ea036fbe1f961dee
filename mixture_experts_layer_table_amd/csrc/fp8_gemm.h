// Tile products of E4M3 operands with one fp32 scale per 128 values of K:
//   out[m][n] = sum over K-blocks b of sx[m,b] sw[n,b] (sum over k in b of X[m][k] W[n][k])
// on v_mfma_f32_32x32x64_f8f6f4. Both operands are K-contiguous.
//
// The two scales of a K-block change from block to block, so a block's product
// cannot go on in the accumulator: two MFMAs (K = 64 each) make it from zero in
// 16 registers, and 16 fused multiply-adds bring it into the accumulator with its
// scale while the next block tile's MFMAs run. The MFMA computes transposed
// 32 x 32 blocks (rows n, columns m, as in gemm.h): a lane holds one row m, so
// sx is one register per 32 rows, and 4 consecutive columns n four times. The
// multiply-adds take half the matrix cores' time, on the vector unit beside them.
//
// LDS tile rows are the 128 bytes of a K-block, 16-byte chunk c of row r at
// chunk c ^ ((r >> 1) & 7): the 16 lanes that are served together read one chunk
// of 16 consecutive rows, 8 even and 8 odd ones, which then lie on 16 different
// 16-byte bank groups.
#pragma once
#include "gemm.h"
#include "fp8_codec.h"

namespace mok {

typedef int i32x8v_t __attribute__((ext_vector_type(8)));
typedef int i32x4v_t __attribute__((ext_vector_type(4)));

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int NSTAGE_>
struct BlkCfg {
    static constexpr int BM = BM_, BN = BN_, BK = kBlk;
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
    static constexpr int NW = WAVES_M * WAVES_N, NT = 64 * NW;
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
    static constexpr int FM = WM / 32, FN = WN / 32;
    static constexpr int NSTAGE = NSTAGE_;
    static constexpr int X_BYTES = BM * BK, W_BYTES = BN * BK, STAGE_BYTES = X_BYTES + W_BYTES;
    static constexpr int SC_OFF = NSTAGE * STAGE_BYTES;   // W row scales, one float per tile row and stage
    static constexpr size_t LDS_BYTES = (size_t)SC_OFF + (size_t)NSTAGE * BN * 4;
    static_assert(WM % 32 == 0 && WN == 64, "a wave stores 64 columns");
    static_assert(BN % 128 == 0 && BN / 64 <= NW, "a wave loads the scales of 64 W rows");
};

// Rows of 128-byte K-blocks into an LDS tile: 8 rows an instruction.
template <class C, int ROWS>
struct BlkLoader {
    static constexpr int IPW = ROWS / 8 / C::NW;
    static_assert(IPW >= 2 && IPW % 2 == 0 && ROWS % (16 * C::NW) == 0, "pairs of instructions per wave");
    rsrc_t res;
    uint32_t v[2];      // the lane's offset in even and in odd groups of 8 rows (their chunk orders differ)
    uint32_t ld8, lds0;
    int len, chunk[2];  // bytes of a row's run; the lane's chunk, in bytes

    // base: the tile's first row at the run's first byte; ld: bytes from row to row
    __device__ __forceinline__ void init(const uint8_t *base, uint32_t ld, int nrows, int len_) {
        len = len_;
        res = make_rsrc(base, nrows > 0 && len > 0 ? (uint32_t)(nrows - 1) * ld + (uint32_t)len : 0u);
        const int wave = wave_id(), L = threadIdx.x & 63;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            chunk[p] = ((L & 7) ^ ((p * 4 + (L >> 4)) & 7)) * 16;   // (row >> 1) & 7 of row 8 i + L / 8, i of parity p
            v[p] = (uint32_t)(wave * IPW * 8 + (L >> 3)) * ld + (uint32_t)chunk[p];
        }
        ld8 = ld * 8;
        lds0 = (uint32_t)(wave * IPW * 1024);
    }
    __device__ __forceinline__ void issue(int kt, uint32_t tile) const {
        const int k0 = kt * kBlk;
        uint32_t o[2] = {v[0], v[1]};
        if (__builtin_expect(k0 + kBlk > len, 0)) {   // what lies behind the run's end is another row's: zeros instead
            asm volatile("");
#pragma unroll
            for (int p = 0; p < 2; ++p) o[p] = k0 + chunk[p] < len ? v[p] : kOutOfRange;
        }
#pragma unroll
        for (int i = 0; i < IPW; ++i)
            load_lds16(res, o[i & 1], (uint32_t)k0 + (uint32_t)i * ld8, tile + lds0 + (uint32_t)(i * 1024));
    }
};

// MFMA operand of 32 tile rows for half s (64 values) of the K-block: lane l
// holds row l % 32, chunks 4 s + 2 (l / 32) and the next one. (The order of k
// inside an MFMA does not matter as long as both operands share it.)
struct BlkFrag {
    i32x8v_t h[2];
};
struct FragAt {       // the lane's four chunk offsets inside 32 rows
    uint32_t o[4];
    __device__ __forceinline__ void init() {
        const int l = threadIdx.x & 63, r = l & 31;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = (i >> 1) * 4 + (l >> 5) * 2 + (i & 1);
            o[i] = (uint32_t)(r * kBlk + ((c ^ ((r >> 1) & 7)) << 4));
        }
    }
};
__device__ __forceinline__ BlkFrag read_frag(const FragAt &at, uint32_t tile) {
    typedef __attribute__((address_space(3))) i32x4v_t lds4_t;
    BlkFrag f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const i32x4v_t lo = *(const lds4_t *)(uintptr_t)(tile + at.o[2 * s]);
        const i32x4v_t hi = *(const lds4_t *)(uintptr_t)(tile + at.o[2 * s + 1]);
        f.h[s] = i32x8v_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
    return f;
}
// Product of a K-block of two 32-row fragments, from zero.
// EXACT false: the fp8 matrix cores. They add 16 products at a time and cut each
// at 2^-13 of the binade of the largest (measured: of 2^16 + 2^e in one group, e = 3
// is kept and e = 2 is lost; groups and blocks are joined in fp32). That is
// 1.5e-5 of a sum's norm for normal values: under a bf16 result's rounding
// (2^-8), but not under an fp32 result's.
// EXACT true, for fp32 results: the same values on the bf16 matrix cores, where
// E4M3 is exact and sums keep fp32 (2e-8 measured), at half the rate.
__device__ __forceinline__ bf16x8_t as_bf16(int lo, int hi) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.0f, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.0f, true);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.0f, false);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.0f, true);
    return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
template <bool EXACT>
__device__ __forceinline__ f32x16_t blk_product(const BlkFrag &w, const BlkFrag &x) {
    f32x16_t t = {};
    if constexpr (EXACT) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const i32x8v_t &a = w.h[i >> 2], &b = x.h[i >> 2];
            const int j = (i & 3) * 2;
            t = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(a[j], a[j + 1]), as_bf16(b[j], b[j + 1]), t, 0, 0, 0);
        }
    } else {
        t = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w.h[0], x.h[0], t, 0, 0, 0, 0, 0, 0);
        t = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w.h[1], x.h[1], t, 0, 0, 0, 0, 0, 0);
    }
    return t;
}

}  // namespace mok
