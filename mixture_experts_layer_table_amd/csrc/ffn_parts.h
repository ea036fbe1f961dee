// Pieces of the gated feed-forward block that its BF16 and MXFP8 kernels
// share: the tile order of a dense product, the fp32 partials of a product
// split over its contraction axis, the row epilogue with an addend, the
// weight gradients, and the kernels that join partials.
//
// Rows are dense here: no schedule, no gather and no ring lie between a tile
// and its tensors, so one launch covers a whole product.
#pragma once
#include <atomic>

#include "ffn_plan.h"
#include "layer_parts.h"
#include "mx_codec.h"

namespace mok {
namespace {

static_assert(kXcds == kGridStep, "the plan counts workgroups as the launches do");

// ----------------------------------------------------------------------------- tiles

struct FfnTile {
    int m0, rows;   // first row and valid rows
    int nt;         // n-tile
    int s;          // run of the contraction axis
};

// Tile of workgroup b of a product of T rows: (m-tile, n-tile, run), in the
// order of the segment GEMMs (each XCD walks a contiguous range of groups of
// kGroupM m-tiles), a run counting as one more n-tile: tiles of one run share
// operand slices, tiles of two runs share none.
__device__ __forceinline__ bool ffn_tile(int T, int bm, int n_tiles, int splits, int b, FfnTile &t) {
    const int mtc = (T + bm - 1) / bm, cols = n_tiles * splits, total = mtc * cols;
    const int per = (total + kXcds - 1) / kXcds;
    const int id = (b % kXcds) * per + b / kXcds;
    if (b / kXcds >= per || id >= total) return false;
    const int gsize = kGroupM * cols, grp = id / gsize, first = grp * kGroupM;
    const int gm = min(kGroupM, mtc - first), r = id % gsize, c = r / gm;
    t.m0 = (first + r % gm) * bm;
    t.rows = min(bm, T - t.m0);
    t.nt = c % n_tiles;
    t.s = c / n_tiles;
    return true;
}
inline unsigned ffn_grid(int64_t T, int bm, int64_t n_tiles, int splits) {
    return (unsigned)(ceil_div(ceil_div(T, bm) * n_tiles * splits, kXcds) * kXcds);
}

// ----------------------------------------------------------------------------- epilogues

__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d) {
    return make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

__device__ __forceinline__ void bstore16(brsrc_t r, uint32_t voff, float a, float b, float c, float d) {
    typedef uint32_t v4u __attribute__((ext_vector_type(4)));
    const v4u w = {__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d)};
    __builtin_amdgcn_raw_buffer_store_b128(w, r, (int)voff, 0, 0);
}

// fp32 partials of one tile, straight from the accumulators: 4 consecutive
// columns per lane. rows: the run's partial rows from the tile's first row on
// (`nrows` valid, ld floats each); col(fn): first column of the wave's fn-th
// 32-column block, every column of the wave valid when `live`.
template <class C, class Col>
__device__ __forceinline__ void store_partials(const f32x16_t (&acc)[C::FM][C::FN], float *rows, int64_t ld, int nrows,
                                               int wm, bool live, Col col) {
    const int lane = epi_lane();
    const brsrc_t dst = rows_rsrc(rows, live ? (uint32_t)((int64_t)nrows * ld * 4) : 0u);
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm) {
        const uint32_t r = (uint32_t)(wm * C::WM + fm * 32 + (lane & 31)) * (uint32_t)(ld * 4);
#pragma unroll
        for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
            for (int g4 = 0; g4 < 4; ++g4)
                bstore16(dst, r + (uint32_t)(col(fn) + g4 * 8 + (lane >> 5) * 4) * 4u, acc[fm][fn][g4 * 4],
                         acc[fm][fn][g4 * 4 + 1], acc[fm][fn][g4 * 4 + 2], acc[fm][fn][g4 * 4 + 3]);
    }
}

// out = addend + acc as bf16 rows through the wave's FragStage area, one
// rounding: the addend's rows are staged first and added in fp32. Both
// descriptors cover the tile's valid rows from the wave's first column on (an
// empty one reads zeros and stores nothing). Output and addend may be one
// buffer: an element is read and written by the same wave, in that order.
template <class C, size_t LDS_END>
__device__ __forceinline__ void store_rows_add(const f32x16_t (&acc)[C::FM][C::FN], int wm, brsrc_t dst, brsrc_t add,
                                               uint32_t row_bytes) {
    using FS = FragStage<C, LDS_END>;
    const int lane = epi_lane();
    const uint32_t area = FS::area(wave_id(), 1);
    const uint32_t v0 = (uint32_t)(wm * C::WM + FS::pass_row(0, lane)) * row_bytes + 2u * (uint32_t)FS::pass_col(lane);
    auto voff = [&](int fm, int p) { return v0 + (uint32_t)(fm * 32 + p * FS::RPP) * row_bytes; };
    uint2 ad[FS::PASSES];
    auto load = [&](int fm) {
#pragma unroll
        for (int p = 0; p < FS::PASSES; ++p) ad[p] = bload8(add, voff(fm, p), 0);
    };
    load(0);
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm) {
#pragma unroll
        for (int p = 0; p < FS::PASSES; ++p) FS::put(area + FS::pass_off(p, lane), ad[p]);
        __builtin_amdgcn_sched_barrier(0);   // phases stay in order: keeps live ranges short
#pragma unroll
        for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
            for (int g4 = 0; g4 < 4; ++g4) {
                const uint32_t o = area + FS::frag_off(fn, g4, lane);
                const uint2 b = FS::get(o);
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = acc[fm][fn][g4 * 4 + j] + bf16_at(b, j);
                FS::put(o, pack4(y[0], y[1], y[2], y[3]));
            }
        __builtin_amdgcn_sched_barrier(0);
        if (fm + 1 < C::FM) load(fm + 1);   // ahead of this fragment's stores: other rows, so also in place
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int p = 0; p < FS::PASSES; ++p) bstore8_nt(dst, voff(fm, p), 0, FS::get(area + FS::pass_off(p, lane)));
    }
}

// The epilogue of a product whose rows are [T][N] bf16 outputs: partials, or out = addend + acc.
template <class C, size_t LDS_END>
__device__ __forceinline__ void dense_epilogue(const f32x16_t (&acc)[C::FM][C::FN], const FfnTile &t, int T, int N,
                                               int splits, int wm, int wn, const uint16_t *addend, uint16_t *out,
                                               float *part) {
    const int nb = t.nt * C::BN + wn * C::WN;
    const bool live = nb < N;   // N % 64 == 0: the wave's columns are all valid or all past N
    if (splits > 1) {
        store_partials<C>(acc, part + ((int64_t)t.s * T + t.m0) * N, N, t.rows, wm, live,
                          [&](int fn) { return nb + fn * 32; });
        return;
    }
    const uint32_t row_bytes = 2u * (uint32_t)N;
    const int64_t o = (int64_t)t.m0 * N + (live ? nb : 0);
    const uint32_t bytes = live ? (uint32_t)t.rows * row_bytes : 0u;
    const brsrc_t dst = rows_rsrc(out + o, bytes);
    if (addend)
        store_rows_add<C, LDS_END>(acc, wm, dst, rows_rsrc(addend + o, bytes), row_bytes);
    else
        staged_rows<C, LDS_END>([&](int fm, int fn, int g4, int j) { return acc[fm][fn][g4 * 4 + j]; }, dst,
                                [&](int fm, int r) -> uint32_t {
                                    return (uint32_t)(wm * C::WM + fm * 32 + r) * row_bytes;
                                });
}

// ----------------------------------------------------------------------------- weight gradients

// out[m][n] = sum over the T rows of X[t][m] * Y[t][n]: X and Y row-major with
// ldx, ldy columns. Columns [0, n0cols) go to out0, the rest to out1 (gate |
// up), both with ldo columns.
struct FfnWgradArgs {
    int T, M, N, n0cols, ldo;
    const uint16_t *x, *y;
    uint16_t *out0, *out1;
};

template <class Cfg>
struct FfnWgrad {
    using C = Cfg;
    using Args = FfnWgradArgs;
    static constexpr bool X_TRANS = true, W_TRANS = true;
    TransLoader<C, C::BM> xl;
    TransLoader<C, C::BN> wl;
    static constexpr int LOADS_PER_STAGE = TransLoader<C, C::BM>::IPW + TransLoader<C, C::BN>::IPW;
    int m0, n0, nk;
    Args a;
    __device__ int mvalid() const { return a.M - m0; }

    // groups of kGroupM m-tiles x all n-tiles, workgroups round-robin over the XCDs
    __device__ bool setup(const Args &args, int b) {
        a = args;
        const int gx = (a.N + C::BN - 1) / C::BN, gy = (a.M + C::BM - 1) / C::BM;
        if (b >= gx * gy) return false;
        const int gsize = kGroupM * gx, g = b / gsize, first = g * kGroupM;
        const int gm = min(kGroupM, gy - first), r = b - g * gsize;
        m0 = (first + r % gm) * C::BM;
        n0 = r / gm * C::BN;
        xl.init(a.x + m0, a.M, a.T, a.M - m0);
        wl.init(a.y + n0, a.N, a.T, a.N - n0);
        nk = (a.T + C::BK - 1) / C::BK;
        return true;
    }
    __device__ void issue(int kt, uint32_t tile) {
        xl.issue(kt * C::BK, tile);
        wl.issue(kt * C::BK, tile + C::X_BYTES);
    }
    __device__ int wrow(int wn, int fn) const { return wn * C::WN + fn * 32; }
    __device__ void epilogue(f32x16_t (&acc)[C::FM][C::FN], int wm, int wn) {
        const int nb = n0 + wn * C::WN;
        if (nb >= a.N) return;   // widths are multiples of 64: the wave's columns are all in one output or all past N
        uint16_t *base = nb < a.n0cols ? a.out0 + nb : a.out1 + (nb - a.n0cols);
        const uint32_t row_bytes = 2u * (uint32_t)a.ldo;
        staged_rows<C, C::LDS_BYTES>([&](int fm, int fn, int g4, int j) { return acc[fm][fn][g4 * 4 + j]; },
                                     rows_rsrc(base, (uint32_t)a.M * row_bytes), [&](int fm, int r) -> uint32_t {
                                         return (uint32_t)(m0 + wm * C::WM + fm * 32 + r) * row_bytes;
                                     });
    }
};
inline unsigned wgrad_grid(int M, int N, int bm) {
    return (unsigned)(ceil_div(ceil_div(M, bm) * ceil_div(N, kTileN), kXcds) * kXcds);
}

// ----------------------------------------------------------------------------- joining partials

// Sum of the runs' partials of 4 consecutive columns, in ascending order. A
// join of few rows is bound by the latency of these loads (each was written by
// another XCD, so none hits in L2): 8 are in flight before the first is added.
// Runs past the last are loaded again and left out of the sum.
constexpr int kJoinBatch = 8;
__device__ __forceinline__ f32x4_t sum_runs(const float *part, int64_t stride, int splits) {
    f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i0 = 0; i0 < splits; i0 += kJoinBatch) {
        f32x4_t v[kJoinBatch];
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j)
            v[j] = *reinterpret_cast<const f32x4_t *>(part + min(i0 + j, splits - 1) * stride);
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j)
            if (i0 + j < splits) s += v[j];
    }
    return s;
}

// 4 codes of a 32-block held by 8 neighbouring lanes (4 values each); every
// lane of the 8 takes part. Returns the codes; `scale` gets the block's byte.
__device__ __forceinline__ uint32_t quantize_lane4(const float (&v)[4], uint32_t &scale) {
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int off = 1; off <= 4; off <<= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off));
    scale = mx_scale_byte_f32(amax);
    const float q = mx_pow2_neg((int)scale - 127);
    return mx_nan_f32(amax) | e4m3x2_scaled(v[0] * q, v[1] * q) | (e4m3x2_scaled(v[2] * q, v[3] * q) << 16);
}

// MXFP8 rows that the block quantizes itself (a, dy, dh) are K-tiled: blocks of 64
// columns, each [T][64], one after the other, so that a K-step of a tile's rows
// is one contiguous run of whole lines; row-major, as the caller's x has to be,
// a step is a 64-byte piece of each row. The operand loads bound these products
// (16,384 x 7,168 x 2,048: forward 700 -> 687 us, backward 1,896 -> 1,876; some
// hundred rows 0.3 us slower). The scales are row-major, [T][columns / 32].
__device__ __forceinline__ uint32_t tiled_at(uint32_t T, uint32_t t, uint32_t k) {   // below T * columns < 2^30
    return (k / 64 * T + t) * 64 + k % 64;
}

// h = sum of the gate/up partials; a = silu(h_g) h_u, as the down product
// reads it: K-tiled, bf16 [I/32][T][32] or MXFP8 [I/64][T][64] with scales.
template <bool MX>
__global__ __launch_bounds__(256) void ffn_join_act(const float *__restrict__ part, int splits, int T, int I,
                                                    uint16_t *__restrict__ h, uint16_t *__restrict__ a,
                                                    uint8_t *__restrict__ aq, uint8_t *__restrict__ aqs) {
    const uint32_t per = (uint32_t)I / 4, idx = blockIdx.x * 256u + threadIdx.x;   // T * I < 2^29
    if (idx >= (uint32_t)T * per) return;   // whole groups of 8 lanes: I / 4 is a multiple of 8
    const int64_t t = idx / per;
    const int i = (int)(idx % per) * 4;
    const int64_t stride = (int64_t)T * 2 * I;
    const float *p = part + t * 2 * I + i;
    const f32x4_t g = sum_runs(p, stride, splits), u = sum_runs(p + I, stride, splits);
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = g[j] * sigmoidf_(g[j]) * u[j];
    if (h) {
        *reinterpret_cast<uint2 *>(h + t * 2 * I + i) = pack4(g[0], g[1], g[2], g[3]);
        *reinterpret_cast<uint2 *>(h + t * 2 * I + I + i) = pack4(u[0], u[1], u[2], u[3]);
    }
    if constexpr (MX) {
        uint32_t sc;
        const uint32_t code = quantize_lane4(v, sc);
        *reinterpret_cast<uint32_t *>(aq + tiled_at((uint32_t)T, (uint32_t)t, (uint32_t)i)) = code;
        if (i % 32 == 0) aqs[(t * I + i) / 32] = (uint8_t)sc;
    } else {
        *reinterpret_cast<uint2 *>(a + ((int64_t)(i / 32) * T + t) * 32 + i % 32) =
            pack4(v[0], v[1], v[2], v[3]);
    }
}

// out = addend + sum of the partials. out and addend may be one buffer.
__global__ __launch_bounds__(256) void ffn_join_out(const float *__restrict__ part, int splits, int T, int N,
                                                    const uint16_t *addend, uint16_t *out) {
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (idx >= (int64_t)T * (N / 4)) return;
    uint2 b = make_uint2(0, 0);
    if (addend) b = reinterpret_cast<const uint2 *>(addend)[idx];
    const f32x4_t s = sum_runs(part + idx * 4, (int64_t)T * N, splits);
    reinterpret_cast<uint2 *>(out)[idx] =
        pack4(s[0] + bf16_at(b, 0), s[1] + bf16_at(b, 1), s[2] + bf16_at(b, 2), s[3] + bf16_at(b, 3));
}

// SwiGLU backward of one value: da arrives, h_g and h_u are the saved rows.
struct GluGrad {
    float a, dg, du;
};
__device__ __forceinline__ GluGrad glu_backward(float da, float hg, float hu) {
    const float s = sigmoidf_(hg), sl = hg * s;
    return GluGrad{sl * hu, da * hu * s * (1.0f + hg * (1.0f - s)), da * sl};
}

// dh and a from the partials of da = dy W_down^T and the saved h.
template <bool MX>
__global__ __launch_bounds__(256) void ffn_join_da(const float *__restrict__ part, int splits, int T, int I,
                                                   const uint16_t *__restrict__ h, uint16_t *__restrict__ dh,
                                                   uint16_t *__restrict__ a, uint8_t *__restrict__ dhq,
                                                   uint8_t *__restrict__ dhqs) {
    const uint32_t per = (uint32_t)I / 4, idx = blockIdx.x * 256u + threadIdx.x;
    if (idx >= (uint32_t)T * per) return;
    const int64_t t = idx / per;
    const int i = (int)(idx % per) * 4;
    const int64_t row = t * 2 * I;
    const uint2 hg = *reinterpret_cast<const uint2 *>(h + row + i);
    const uint2 hu = *reinterpret_cast<const uint2 *>(h + row + I + i);
    const f32x4_t s = sum_runs(part + t * I + i, (int64_t)T * I, splits);
    float va[4], vg[4], vu[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const GluGrad r = glu_backward(s[j], bf16_at(hg, j), bf16_at(hu, j));
        va[j] = r.a;
        vg[j] = r.dg;
        vu[j] = r.du;
    }
    auto put = [](uint16_t *p, const float (&v)[4]) {
        *reinterpret_cast<uint2 *>(p) = pack4(v[0], v[1], v[2], v[3]);
    };
    put(a + t * I + i, va);
    put(dh + row + i, vg);
    put(dh + row + I + i, vu);
    if constexpr (MX) {
        uint32_t sg, su;
        const uint32_t cg = quantize_lane4(vg, sg), cu = quantize_lane4(vu, su);
        *reinterpret_cast<uint32_t *>(dhq + tiled_at((uint32_t)T, (uint32_t)t, (uint32_t)i)) = cg;
        *reinterpret_cast<uint32_t *>(dhq + tiled_at((uint32_t)T, (uint32_t)t, (uint32_t)(I + i))) = cu;
        if (i % 32 == 0) {
            dhqs[(row + i) / 32] = (uint8_t)sg;
            dhqs[(row + I + i) / 32] = (uint8_t)su;
        }
    }
}

inline unsigned join_grid(int64_t T, int64_t N) { return (unsigned)ceil_div(T * (N / 4), 256); }

// ----------------------------------------------------------------------------- launches

// Dynamic LDS above 64 KiB has to be allowed once per kernel and device.
template <class K>
hipError_t allow_lds(K *kernel, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    const hipError_t r =
        hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (r == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return r;
}

}  // namespace
}  // namespace mok
