// Products on operands in blocks of 128 (fp8_gemm.h): rows by weights, dense or
// grouped by expert, and the weight gradients.
#include <atomic>

#include "fp8_gemm.h"
#include "fp8_plan.h"
#include "layer_parts.h"

namespace mok {
namespace {

using CfgL = BlkCfg<256, 256, 2, 4, 2>;
using CfgM = BlkCfg<128, 256, 2, 4, 2>;

struct BlkArgs {
    int64_t xs_ld, ws_ld;    // entries from one block's scales to the next (X; W by rows)
    const uint8_t *x, *w;
    const float *xs, *ws;
    const int32_t *offsets;  // NULL: one product
    const void *addend;
    void *out;
    int M, N, K, E;          // output rows (of all experts together, or of one), columns, contraction
    int ldx, ldw;            // bytes from row to row
};

// One tile: output rows [m0, m0 + rows) x columns [n0, ..), contraction [k0, k0 + len).
struct BlkTile {
    const uint8_t *x, *w;    // first row at k0
    const float *xs, *ws;    // scales of the first row (W by tiles: the first block row) at k0
    int rows, cols, len;
    int64_t out;             // first element in out
};

__device__ __forceinline__ int clamp_row(int v, int M) { return min(max(v, 0), M); }

// ----------------------------------------------------------------------------- tiles

// Number of row tiles of expert e (lane-wise), its first row and its rows.
__device__ __forceinline__ int expert_tiles(const BlkArgs &a, int bm, int e, int &lo, int &n) {
    lo = n = 0;
    if (e < a.E) {
        lo = clamp_row(a.offsets[e], a.M);
        n = max(clamp_row(a.offsets[e + 1], a.M) - lo, 0);
    }
    return (n + bm - 1) / bm;
}
__device__ __forceinline__ int lane_scan(int v) {   // inclusive
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if ((int)(threadIdx.x & 63) >= d) v += o;
    }
    return v;
}
__device__ __forceinline__ int uniform_i(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Row tile and column tile of workgroup b; false: none. As in the segment GEMMs
// each XCD walks a contiguous range of tiles, in groups of kGroupM row tiles.
struct RowTile {
    int e, m0, rows, nt;
};
__device__ __forceinline__ bool locate(const BlkArgs &a, int bm, int n_tiles, int b, RowTile &t) {
    int total = (a.M + bm - 1) / bm;
    const int lane = threadIdx.x & 63;
    if (a.E > 0) {
        total = 0;
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            int lo, n;
            total += __shfl(lane_scan(expert_tiles(a, bm, e0 + lane, lo, n)), 63);
        }
        total = uniform_i(total);
    }
    const int all = total * n_tiles, per = (all + kXcds - 1) / kXcds, id = (b % kXcds) * per + b / kXcds;
    if (b / kXcds >= per || id >= all) return false;
    const int gsize = kGroupM * n_tiles, first = id / gsize * kGroupM, gm = min(kGroupM, total - first), r = id % gsize;
    const int mt = first + r % gm;
    t.nt = r / gm;
    if (a.E == 0) {
        t.e = 0;
        t.m0 = mt * bm;
        t.rows = min(bm, a.M - t.m0);
        return true;
    }
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        int lo, n;
        const int c = expert_tiles(a, bm, e0 + lane, lo, n), incl = before + lane_scan(c);
        const uint64_t past = __ballot(incl > mt);
        if (past) {
            const int who = __builtin_ctzll(past);
            const int i = mt - __shfl(incl - c, who);
            t.e = uniform_i(e0 + who);
            t.m0 = uniform_i(__shfl(lo, who) + i * bm);
            t.rows = uniform_i(min(bm, __shfl(n, who) - i * bm));
            return true;
        }
        before = __shfl(incl, 63);
    }
    return false;
}

// ----------------------------------------------------------------------------- the tile's product

// WROWS: W has a scale per row and block (weight gradients), else per 128 rows and
// block. F32: fp32 results, whose products are exact (blk_product).
template <class C, bool WROWS, bool F32>
__device__ __forceinline__ void blk_tile(const BlkArgs &a, const BlkTile &t, uint32_t lds) {
    constexpr int FM = C::FM, FN = C::FN;
    const int wave = wave_id(), wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
    const int lane = threadIdx.x & 63;
    const int nk = uniform_i((t.len + kBlk - 1) / kBlk);
    f32x16_t acc[FM][FN];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[fm][fn][r] = 0.0f;

    BlkLoader<C, C::BM> xl;
    BlkLoader<C, C::BN> wl;
    xl.init(t.x, (uint32_t)a.ldx, t.rows, t.len);
    wl.init(t.w, (uint32_t)a.ldw, t.cols, t.len);
    FragAt at;
    at.init();
    const uint32_t xs_off = (uint32_t)(wm * C::WM + (lane & 31)) * 4u;
    const float *ws_tile = t.ws;   // scales of the wave's 128 W rows, one per block
    if constexpr (!WROWS) ws_tile += (int64_t)min(wn * 64 / kBlk, (t.cols - 1) / kBlk) * a.ws_ld;

    float sx[FM], sx_next[FM], sw_lane = 0.0f;
    auto stage = [&](int kt) { return lds + (uint32_t)((kt % C::NSTAGE) * C::STAGE_BYTES); };
    auto w_scales = [&](int kt) { return lds + (uint32_t)(C::SC_OFF + (kt % C::NSTAGE) * C::BN * 4); };
    auto issue = [&](int kt) {
        const uint32_t st = stage(kt);
        xl.issue(kt, st);
        wl.issue(kt, st + C::X_BYTES);
        if constexpr (WROWS) {
            if (wave < C::BN / 64)
                load_lds4(make_rsrc(t.ws + (int64_t)kt * a.ws_ld, (uint32_t)t.cols * 4u),
                          (uint32_t)(wave * 64 + lane) * 4u, 0, w_scales(kt) + (uint32_t)wave * 256u);
        }
    };
    auto load_sx = [&](int kt, float (&s)[FM]) {
        const brsrc_t r = rows_rsrc(t.xs + (int64_t)kt * a.xs_ld, (uint32_t)t.rows * 4u);
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
            s[fm] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)(xs_off + (uint32_t)fm * 128u), 0, 0));
    };
    if (nk > 0) {
        issue(0);
        load_sx(0, sx);
    }
    for (int kt = 0; kt < nk; ++kt) {
        wait_vmcnt<0>();
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) asm volatile("" : "+v"(sx[fm]));
        lds_barrier();   // block kt has landed, and no wave reads block kt - 1 any more
        if constexpr (!WROWS) {
            if (kt % 64 == 0) {   // the next 64 blocks' scales, one a lane
                sw_lane = ws_tile[min(kt + lane, nk - 1)];
                asm volatile("" : "+v"(sw_lane));
            }
        }
        if (kt + 1 < nk) {
            issue(kt + 1);
            load_sx(kt + 1, sx_next);
        }
        const uint32_t st = stage(kt);
        BlkFrag w[FN];
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) w[fn] = read_frag(at, st + (uint32_t)(C::X_BYTES + (wn * 64 + fn * 32) * kBlk));
        float s[FM];
        if constexpr (!WROWS) {
            const float sw = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(sw_lane), kt % 64));
#pragma unroll
            for (int fm = 0; fm < FM; ++fm) s[fm] = sx[fm] * sw;
        }
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            const BlkFrag x = read_frag(at, st + (uint32_t)((wm * C::WM + fm * 32) * kBlk));
#pragma unroll
            for (int fn = 0; fn < FN; ++fn) {
                const f32x16_t p = blk_product<F32>(w[fn], x);
                if constexpr (WROWS) {
                    const uint32_t sa = w_scales(kt) + (uint32_t)(wn * 64 + fn * 32 + (lane >> 5) * 4) * 4u;
#pragma unroll
                    for (int g4 = 0; g4 < 4; ++g4) {
                        const f32x4_t sw = *(const __attribute__((address_space(3))) f32x4_t *)(uintptr_t)(sa + g4 * 32);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[fm][fn][g4 * 4 + j] =
                                __builtin_fmaf(p[g4 * 4 + j], sx[fm] * sw[j], acc[fm][fn][g4 * 4 + j]);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[fm][fn][r] = __builtin_fmaf(p[r], s[fm], acc[fm][fn][r]);
                }
            }
        }
        wait_lgkm0();
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) sx[fm] = sx_next[fm];
    }
    lds_barrier();   // the waves' staging areas lie where blocks were

    // out = addend + acc: rows through the wave's staging area (bf16), or 16 bytes a lane (fp32)
    const int c0 = wn * 64, el = epi_lane();
    const int valid = min(t.cols - c0, 64);   // a multiple of 16
    constexpr uint32_t es = F32 ? 4u : 2u;
    const uint32_t row_bytes = (uint32_t)a.N * es;
    const int64_t o = t.out + c0;
    const uint32_t bytes = valid > 0 ? (uint32_t)(t.rows - 1) * row_bytes + (uint32_t)valid * es : 0u;
    const int64_t at_byte = (valid > 0 ? o : 0) * es;
    const brsrc_t dst = rows_rsrc(static_cast<char *>(a.out) + at_byte, bytes);
    const brsrc_t add = rows_rsrc(a.addend ? static_cast<const char *>(a.addend) + at_byte : static_cast<char *>(a.out),
                                  a.addend ? bytes : 0u);
    if constexpr (F32) {
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            const uint32_t r = (uint32_t)(wm * C::WM + fm * 32 + (el & 31)) * row_bytes;
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int g4 = 0; g4 < 4; ++g4) {
                    const int c = fn * 32 + g4 * 8 + (el >> 5) * 4;
                    const uint32_t v = c < valid ? r + (uint32_t)c * 4u : kOutOfRange;
                    typedef uint32_t v4u __attribute__((ext_vector_type(4)));
                    v4u w = __builtin_amdgcn_raw_buffer_load_b128(add, (int)v, 0, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = __float_as_uint(acc[fm][fn][g4 * 4 + j] + __uint_as_float(w[j]));
                    __builtin_amdgcn_raw_buffer_store_b128(w, dst, (int)v, 0, 0);
                }
        }
    } else {
        using FS = FragStage<C, C::LDS_BYTES>;
        const uint32_t area = FS::area(wave, 1);
        const int col = FS::pass_col(el);
        const uint32_t v0 = col < valid
                                ? (uint32_t)(wm * C::WM + FS::pass_row(0, el)) * row_bytes + 2u * (uint32_t)col
                                : kOutOfRange;
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            if (a.addend) {
#pragma unroll
                for (int p = 0; p < FS::PASSES; ++p)
                    FS::put(area + FS::pass_off(p, el), bload8(add, v0 + (uint32_t)(fm * 32 + p * FS::RPP) * row_bytes, 0));
            }
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int g4 = 0; g4 < 4; ++g4) {
                    const uint32_t f = area + FS::frag_off(fn, g4, el);
                    float y[4];
                    const uint2 b = a.addend ? FS::get(f) : make_uint2(0, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = acc[fm][fn][g4 * 4 + j] + bf16_at(b, j);
                    FS::put(f, make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])));
                }
#pragma unroll
            for (int p = 0; p < FS::PASSES; ++p)
                bstore8_nt(dst, v0 + (uint32_t)(fm * 32 + p * FS::RPP) * row_bytes, 0, FS::get(area + FS::pass_off(p, el)));
        }
    }
}

template <class C, bool F32>
__global__ __launch_bounds__(C::NT, 2) void blk_matmul(BlkArgs a) {
    extern __shared__ __attribute__((aligned(1024))) char lds_raw[];
    const int n_tiles = (a.N + C::BN - 1) / C::BN;
    RowTile r;
    if (!locate(a, C::BM, n_tiles, (int)blockIdx.x, r)) return;
    const int n0 = r.nt * C::BN, nb = (a.N + kBlk - 1) / kBlk, kb = (a.K + kBlk - 1) / kBlk;
    BlkTile t;
    t.x = a.x + (int64_t)r.m0 * a.K;
    t.w = a.w + ((int64_t)r.e * a.N + n0) * a.K;
    t.xs = a.xs + r.m0;
    t.ws = a.ws + ((int64_t)r.e * nb + n0 / kBlk) * kb;
    t.rows = r.rows;
    t.cols = min(C::BN, a.N - n0);
    t.len = a.K;
    t.out = (int64_t)r.m0 * a.N + n0;
    blk_tile<C, false, F32>(a, t, (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds_raw);
}

// Weight gradients: rows of `x` are those of dy (output rows), rows of `w` those of x (columns).
template <class C, bool F32>
__global__ __launch_bounds__(C::NT, 2) void blk_wgrad(BlkArgs a) {
    extern __shared__ __attribute__((aligned(1024))) char lds_raw[];
    const int gx = (a.N + C::BN - 1) / C::BN, gy = (a.M + C::BM - 1) / C::BM;
    const int per = (gx * gy + kXcds - 1) / kXcds * kXcds;   // workgroups of an expert
    const int e = (int)blockIdx.x / per, b = (int)blockIdx.x % per;
    const int id = (b % kXcds) * (per / kXcds) + b / kXcds;
    if (id >= gx * gy) return;
    const int gsize = kGroupM * gx, first = id / gsize * kGroupM, gm = min(kGroupM, gy - first), r = id % gsize;
    const int m0 = (first + r % gm) * C::BM, n0 = r / gm * C::BN;
    int r0 = 0, r1 = a.K;
    if (a.E > 0) {
        r0 = uniform_i(clamp_row(a.offsets[e], a.K)) & ~(kBlk - 1);
        r1 = uniform_i(clamp_row(a.offsets[e + 1], a.K));
    }
    BlkTile t;
    t.x = a.x + (int64_t)m0 * a.ldx + r0;
    t.w = a.w + (int64_t)n0 * a.ldw + r0;
    t.xs = a.xs + (int64_t)(r0 / kBlk) * a.xs_ld + m0;
    t.ws = a.ws + (int64_t)(r0 / kBlk) * a.ws_ld + n0;
    t.rows = min(C::BM, a.M - m0);
    t.cols = min(C::BN, a.N - n0);
    t.len = max(r1 - r0, 0);
    t.out = ((int64_t)e * a.M + m0) * a.N + n0;
    blk_tile<C, true, F32>(a, t, (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds_raw);
}

template <class K>
hipError_t allow_lds(K *kernel, size_t bytes, std::atomic<uint64_t> &done) {   // once per kernel and device
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

template <class C, bool F32>
hipError_t launch_matmul(const BlkArgs &a, hipStream_t st) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds(blk_matmul<C, F32>, C::LDS_BYTES, done);
    if (e != hipSuccess) return e;
    // row tiles: at most one more for each expert that has rows
    const int64_t mt = ceil_div(a.M, C::BM) + (a.E > 0 ? std::min(a.E, a.M) : 0);
    const int64_t grid = ceil_div(mt * ceil_div(a.N, C::BN), kXcds) * kXcds;
    KernelTimer tm("fp8_matmul", st);
    blk_matmul<C, F32><<<(unsigned)grid, C::NT, C::LDS_BYTES, st>>>(a);
    return hipGetLastError();
}

template <class C, bool F32>
hipError_t launch_wgrad(const BlkArgs &a, hipStream_t st) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds(blk_wgrad<C, F32>, C::LDS_BYTES, done);
    if (e != hipSuccess) return e;
    const int64_t per = ceil_div(ceil_div(a.N, C::BN) * ceil_div(a.M, C::BM), kXcds) * kXcds;
    const int64_t grid = per * std::max(a.E, 1);
    KernelTimer tm("fp8_wgrad", st);
    blk_wgrad<C, F32><<<(unsigned)grid, C::NT, C::LDS_BYTES, st>>>(a);
    return hipGetLastError();
}

}  // namespace

mok_status launch_fp8_matmul(const BlkPlan &p, void *workspace, const uint8_t *a_elems, const float *a_scales,
                             const uint8_t *b_elems, const float *b_scales, const int32_t *offsets, void *out,
                             hipStream_t st) {
    (void)workspace;
    BlkArgs a{};
    a.xs_ld = p.M;
    a.ws_ld = (p.K + kBlk - 1) / kBlk;
    a.x = a_elems;
    a.w = b_elems;
    a.xs = a_scales;
    a.ws = b_scales;
    a.offsets = offsets;
    a.out = out;
    a.M = (int)p.M;
    a.N = p.N;
    a.K = p.K;
    a.E = p.E;
    a.ldx = a.ldw = p.K;
    hipError_t e;
    if (p.f32) e = launch_matmul<CfgM, true>(a, st);
    else e = p.bm == CfgM::BM ? launch_matmul<CfgM, false>(a, st) : launch_matmul<CfgL, false>(a, st);
    return check_hip(e, "mok_fp8_matmul");
}

mok_status launch_fp8_wgrad(const BlkPlan &p, void *workspace, const uint8_t *dy_elems, const float *dy_scales,
                            const uint8_t *x_elems, const float *x_scales, const int32_t *offsets, const void *addend,
                            void *out, hipStream_t st) {
    (void)workspace;
    BlkArgs a{};
    a.xs_ld = p.N;
    a.ws_ld = p.K;
    a.x = dy_elems;
    a.w = x_elems;
    a.xs = dy_scales;
    a.ws = x_scales;
    a.offsets = offsets;
    a.addend = addend;
    a.out = out;
    a.M = p.N;
    a.N = p.K;
    a.K = (int)p.M;
    a.E = p.E;
    a.ldx = a.ldw = (int)p.M;
    hipError_t e;
    if (p.f32) e = launch_wgrad<CfgM, true>(a, st);
    else e = p.bm == CfgM::BM ? launch_wgrad<CfgM, false>(a, st) : launch_wgrad<CfgL, false>(a, st);
    return check_hip(e, "mok_fp8_wgrad");
}

}  // namespace mok
