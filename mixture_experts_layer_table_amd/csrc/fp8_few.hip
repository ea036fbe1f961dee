// Products of few rows by weights in blocks of 128 (mok_fp8_matmul): the weights
// are read once, straight into registers, and bound the time.
//
// A workgroup takes 16 or 32 rows of W (of one expert) over the whole contraction, its 8
// waves K-blocks in turn, so that together they read whole runs of the rows. A
// wave holds one K-block: 16 rows x 128 bytes, two 16-byte loads a lane, and the
// same of up to 16 MT rows of X (rows past the last read as zeros).
// v_mfma_f32_16x16x128_f8f6f4 (rows n, columns m) makes a block's product from
// zero; the scales join it to the accumulator as in fp8_gemm.h, and the waves' sums
// are added through LDS in order.
//
// One block a wave keeps the registers few (MT = 1: 40), so that four workgroups
// share a compute unit and their loads overlap; seven blocks in flight a wave took
// the same time for one round of workgroups (1 row x 4,096 x 7,168: 7.9 against 7.8
// us, 3.8 TB/s with its launch) and 124 against 46 us for 28 rounds of short rows (16
// experts of one row each, 7,168 x 2,048; 42 and 5.6 TB/s with 32 rows of W a
// workgroup). Past some 16 rows X's bytes from L2, once for each workgroup, bound it.
#include "fp8_plan.h"
#include "fp8_tiles.h"

namespace mok {
namespace {

constexpr int kFewWaves = 8;

template <bool EXACT>
__device__ __forceinline__ f32x4_t few_product(const i32x8v_t &w, const i32x8v_t &x) {
    f32x4_t t = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (EXACT) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(w[2 * i], w[2 * i + 1]),
                                                        as_bf16(x[2 * i], x[2 * i + 1]), t, 0, 0, 0);
    } else {
        t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, t, 0, 0, 0, 0, 0, 0);
    }
    return t;
}

typedef uint32_t u32x4v_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x8v_t load_block(brsrc_t r, uint32_t lo, uint32_t hi, uint32_t soff) {
    const u32x4v_t a = __builtin_amdgcn_raw_buffer_load_b128(r, (int)lo, (int)soff, 0);
    const u32x4v_t b = __builtin_amdgcn_raw_buffer_load_b128(r, (int)hi, (int)soff, 0);
    return i32x8v_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// MT: tiles of 16 rows of X at a time; NW: of 16 rows of W.
template <int MT, int NW, bool F32>
__global__ __launch_bounds__(64 * kFewWaves) void blk_few(BlkArgs a) {
    __shared__ __attribute__((aligned(16))) float red[kFewWaves][MT * 16][NW * 16];
    const int strips = (a.N / 16 + NW - 1) / NW, n0 = (int)blockIdx.x % strips * 16 * NW;
    const int cols = min(a.N - n0, 16 * NW);
    // the i-th expert that has rows
    const Found f = find_tile(a, (int)blockIdx.x / strips, [](int n) { return n > 0 ? 1 : 0; });
    if (f.e < 0) return;
    const int e = f.e, lo = f.lo, hi = lo + f.n;
    const int wave = wave_id(), lane = threadIdx.x & 63, row = lane & 15, q = lane >> 4;
    const int nk = (a.K + kBlk - 1) / kBlk, nb = (a.N + kBlk - 1) / kBlk;
    const brsrc_t wr = rows_rsrc(a.w + ((int64_t)e * a.N + n0) * a.K, (uint32_t)cols * (uint32_t)a.K);
    const float *ws = a.ws + ((int64_t)e * nb + n0 / kBlk) * nk;
    const uint32_t own = (uint32_t)row * (uint32_t)a.K + (uint32_t)q * 16u;
    for (int m0 = lo; m0 < hi; m0 += 16 * MT) {
        const int rows = min(hi - m0, 16 * MT);
        const brsrc_t xr = rows_rsrc(a.x + (int64_t)m0 * a.K, (uint32_t)rows * (uint32_t)a.K);
        f32x4_t acc[MT][NW];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < NW; ++n) acc[t][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        for (int kb = wave; kb < nk; kb += kFewWaves) {
            const int at = kb * kBlk;
            // what lies behind a row's end is another row's: zeros instead
            const bool l = at + q * 16 < a.K, h = at + 64 + q * 16 < a.K;
            const auto tile = [&](brsrc_t r, int i) {   // rows 16 i .. of r
                const uint32_t o = own + (uint32_t)i * 16u * (uint32_t)a.K;
                return load_block(r, l ? o : kOutOfRange, h ? o + 64u : kOutOfRange, (uint32_t)at);
            };
            i32x8v_t w[NW], x[MT];
            float sx[MT];
#pragma unroll
            for (int n = 0; n < NW; ++n) w[n] = tile(wr, n);
#pragma unroll
            for (int t = 0; t < MT; ++t) x[t] = tile(xr, t);
            const float sw = ws[kb], *s = a.xs + (int64_t)kb * a.xs_ld + m0;
#pragma unroll
            for (int t = 0; t < MT; ++t) sx[t] = s[min(t * 16 + row, rows - 1)];
            __builtin_amdgcn_sched_barrier(0);   // all of them in flight before the first product
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const float both = sw * sx[t];
#pragma unroll
                for (int n = 0; n < NW; ++n) {
                    const f32x4_t p = few_product<F32>(w[n], x[t]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[t][n][j] = __builtin_fmaf(p[j], both, acc[t][n][j]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < NW; ++n)
                *reinterpret_cast<f32x4_t *>(&red[wave][t * 16 + row][n * 16 + q * 4]) = acc[t][n];
        __syncthreads();
        for (int i = (int)threadIdx.x; i < rows * 8 * NW; i += 64 * kFewWaves) {
            const int m = i / (8 * NW), n = i % (8 * NW) * 2;
            if (n >= cols) continue;   // the last strip of an odd number of tiles
            float u = 0.0f, v = 0.0f;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) {
                u += red[w][m][n];
                v += red[w][m][n + 1];
            }
            const int64_t o = (int64_t)(m0 + m) * a.N + n0 + n;
            if constexpr (F32)
                *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + o) = make_float2(u, v);
            else
                *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + o) = pack_bf16x2(u, v);
        }
        __syncthreads();
    }
}

template <int MT, int NW>
hipError_t launch_few(const BlkArgs &a, bool f32, hipStream_t st) {
    const unsigned grid = (unsigned)((a.N / 16 + NW - 1) / NW) * (unsigned)(a.E > 0 ? std::min(a.E, a.M) : 1);
    KernelTimer tm("fp8_matmul_few", st);
    if (f32)
        blk_few<MT, NW, true><<<grid, 64 * kFewWaves, 0, st>>>(a);
    else
        blk_few<MT, NW, false><<<grid, 64 * kFewWaves, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_blk_few(const BlkArgs &a, int mt, int nw, bool f32, hipStream_t st) {
    if (nw == 1)
        return mt == 1   ? launch_few<1, 1>(a, f32, st)
               : mt == 2 ? launch_few<2, 1>(a, f32, st)
                         : launch_few<4, 1>(a, f32, st);
    return mt == 1   ? launch_few<1, 2>(a, f32, st)
           : mt == 2 ? launch_few<2, 2>(a, f32, st)
                     : launch_few<4, 2>(a, f32, st);
}

}  // namespace mok
