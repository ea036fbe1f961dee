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

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int NSTAGE_, int PER_TILE_, bool EARLY_W_ = false>
struct BlkCfg {
    static constexpr int BM = BM_, BN = BN_, BK = kBlk;
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
    static constexpr int NW = WAVES_M * WAVES_N, NT = 64 * NW;
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
    static constexpr int FM = WM / 32, FN = WN / 32;
    static constexpr int NSTAGE = NSTAGE_;
    static constexpr int X_BYTES = BM * BK, W_BYTES = BN * BK, STAGE_BYTES = X_BYTES + W_BYTES;
    // Scales of one stage: 64 floats from each wave (X rows from the first waves, W rows from the last ones). Their
    // ring is one deeper: those of a block's last tiles are read when its buffer is already being filled.
    static constexpr int SC_BYTES = NW * 256, SC_W = (NW - BN / 64) * 256;
    static constexpr int SC_OFF = NSTAGE * STAGE_BYTES;
    static constexpr size_t LDS_BYTES = (size_t)SC_OFF + (size_t)(NSTAGE + 1) * SC_BYTES;
    static_assert(WM % 32 == 0 && WN == 64, "a wave stores 64 columns");
    static_assert(BM % 128 == 0 && BN % 128 == 0 && BM / 64 + BN / 64 <= NW, "a wave loads 64 rows' scales");
    // Vector-memory loads of a wave and K-block, and how many it issues per tile (see blk_tile)
    static constexpr int LOADS = BM / 8 / NW + BN / 8 / NW + 1, PER_TILE = PER_TILE_;
    static constexpr bool EARLY_W = EARLY_W_;
    static_assert(NSTAGE >= 2 && LDS_BYTES <= 160 * 1024, "two stages at least; LDS of a compute unit");
};

// Rows of 128-byte K-blocks into an LDS tile: 8 rows an instruction. Lane l of
// instruction i brings 16 bytes of row 8 i + l / 8 to place l % 8 of it, so it
// loads chunk (l % 8) ^ ((row >> 1) & 7): the chunks of even and of odd i differ in
// bit 2 alone. One register a lane holds its offset, one its even chunk.
template <class C, int ROWS>
struct BlkLoader {
    static constexpr int IPW = ROWS / 8 / C::NW;
    static_assert(IPW >= 2 && IPW % 2 == 0 && ROWS % (16 * C::NW) == 0, "pairs of instructions per wave");
    rsrc_t res;
    uint32_t ld8, lds0;
    int len;            // bytes of a row's run

    static __device__ __forceinline__ uint32_t lane_chunk() {   // in bytes
        const int L = threadIdx.x & 63;
        return (uint32_t)(((L & 7) ^ (L >> 4)) * 16);
    }
    // The lane's offset from the tile's first row, without its chunk.
    static __device__ __forceinline__ uint32_t lane_row(uint32_t ld) {
        return (uint32_t)(wave_id() * IPW * 8 + (int)((threadIdx.x & 63) >> 3)) * ld;
    }
    // base: the tile's first row at the run's first byte; ld: bytes from row to row, a multiple of 16. A run's last
    // chunk is loaded whole, in the last row too: past a shorter buffer's end nothing of it would come.
    __device__ __forceinline__ void init(const uint8_t *base, uint32_t ld, int nrows, int len_) {
        len = len_;
        res = make_rsrc(base, nrows > 0 && len > 0 ? (uint32_t)(nrows - 1) * ld + (((uint32_t)len + 15u) & ~15u) : 0u);
        ld8 = ld * 8;
        lds0 = (uint32_t)(wave_id() * IPW * 1024);
    }
    // Instruction i of block kt. Without a branch: what lies behind the run's end (or is a block past the last) is
    // another row's, so its lanes read zeros instead.
    __device__ __forceinline__ void issue(int i, int kt, uint32_t tile, uint32_t row, uint32_t chunk) const {
        const int k0 = kt * kBlk;
        const uint32_t c = i % 2 ? chunk ^ 64u : chunk;
        load_lds16(res, k0 + (int)c < len ? row + c : kOutOfRange, (uint32_t)k0 + (uint32_t)i * ld8,
                   tile + lds0 + (uint32_t)(i * 1024));
    }
};

// Zeros behind a run's end in the last 16-byte chunk of its last K-block, in every tile row (len: the run's, no
// multiple of 16). Each lane clears one of the rows that its own wave loaded (X rows in the lower half of the wave, W
// rows in the upper one), so the wave's own wait for its loads is enough before, and the workgroup's barrier after.
template <class C>
__device__ __forceinline__ void clear_behind(uint32_t tile, int len) {
    constexpr int XR = BlkLoader<C, C::BM>::IPW * 8, WR = BlkLoader<C, C::BN>::IPW * 8;
    static_assert(XR <= 32 && WR <= 32, "a row a lane");
    const bool upper = threadIdx.x & 32;
    const int i = threadIdx.x & 31, row = wave_id() * (upper ? WR : XR) + i, c = (len & (kBlk - 1)) / 16;
    if (i < (upper ? WR : XR)) {
        const uint32_t at = tile + (uint32_t)((upper ? C::X_BYTES : 0) + row * kBlk + (c ^ ((row >> 1) & 7)) * 16);
        typedef __attribute__((address_space(3))) uint8_t lds_u8;
        for (int b = len & 15; b < 16; ++b) *(lds_u8 *)(uintptr_t)(at + (uint32_t)b) = 0;
    }
    wait_lgkm0();
}

// MFMA operand of 32 tile rows for half s (64 values) of the K-block: lane l
// holds row l % 32, chunks 4 s + 2 (l / 32) and the next one. (The order of k
// inside an MFMA does not matter as long as both operands share it.)
struct BlkFrag {
    i32x8v_t h[2];
};
// The lane's first chunk inside 32 rows; the others lie at it ^ 16 (the next chunk), ^ 64 (the other half) and ^ 80.
__device__ __forceinline__ uint32_t frag_lane() {
    const int l = threadIdx.x & 63, r = l & 31;
    return (uint32_t)(r * kBlk + (((l >> 5) * 2) ^ ((r >> 1) & 7)) * 16);
}
// Fragment at `at` (a multiple of 128 bytes, and frag_lane() added) + OFF, a constant that goes into the instructions.
template <uint32_t OFF>
__device__ __forceinline__ BlkFrag read_frag(uint32_t at) {
    typedef __attribute__((address_space(3))) i32x4v_t lds4_t;
    typedef __attribute__((address_space(3))) char lds_t;
    BlkFrag f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const i32x4v_t lo = *(const lds4_t *)((const lds_t *)(uintptr_t)(at ^ (uint32_t)(64 * s)) + OFF);
        const i32x4v_t hi = *(const lds4_t *)((const lds_t *)(uintptr_t)(at ^ (uint32_t)(64 * s + 16)) + OFF);
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
