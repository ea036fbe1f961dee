// Products on operands in blocks of 128 (fp8_gemm.h): rows by weights, dense or
// grouped by expert, and the weight gradients.
#include <atomic>

#include "fp8_gemm.h"
#include "fp8_plan.h"
#include "layer_parts.h"

namespace mok {
namespace {

using CfgL = BlkCfg<256, 256, 2, 4, 2, 3, true>;
using CfgM = BlkCfg<128, 256, 2, 4, 3, 3>;

struct BlkArgs {
    int64_t xs_ld, ws_ld;    // entries from one block's scales to the next (X; W by rows)
    const uint8_t *x, *w;
    const float *xs, *ws;
    const int32_t *offsets;  // NULL: one product
    const void *addend;
    void *out;
    int M, N, K, E;          // output rows (of all experts together, or of one), columns, contraction
    int ld;                  // bytes from row to row, of both
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

// x of lane R of the lane's row of 16
template <int R>
__device__ __forceinline__ float lane_of_16(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + R, 0xF, 0xF, true));
}

// acc += p * s, or with a scale per W row (register R's in lane R of 16) acc += p * (s * sw_R)
template <bool WROWS, int... R>
__device__ __forceinline__ void scaled_add(f32x16_t &acc, const f32x16_t &p, float s, float sw,
                                           std::integer_sequence<int, R...>) {
    ((acc[R] = __builtin_fmaf(p[R], WROWS ? s * lane_of_16<R>(sw) : s, acc[R])), ...);
}

// WROWS: W has a scale per row and block (weight gradients), else per 128 rows and
// block. F32: fp32 results, whose products are exact (blk_product).
//
// A wave goes through its FM x FN block tiles of a K-block in row order, one
// tile's MFMAs issued ahead of the previous tile's multiply-adds (two product
// registers in turn), so that the matrix cores run through. X fragments are read
// one row of tiles ahead. One barrier a K-block, ahead of its last row of tiles:
// by then every fragment of block kt is in registers, so its buffer can take block
// kt + NSTAGE; and block kt + 1 has landed, whose first fragments are read during
// that last row. Loads thus have (NSTAGE - 1) K-blocks' time. With two stages
// (EARLY_W) that is short, so a second barrier after the first row frees the W half
// of the buffer, whose fragments a wave holds through the block: its loads go out
// half a block sooner.
// 16,384 x 4,096 x 7,168 on one card: 581 us as a plain loop, 432 with products in
// turn, 401 with the loads in branchless form, 386 with three of a wave's nine loads
// a tile instead of all behind the barrier, 371 with the second barrier; 282 without
// loads and multiply-adds, where the clock (1.9 GHz) is the limit.
template <class C, bool WROWS, bool F32>
__device__ __forceinline__ void blk_tile(const BlkArgs &a, const BlkTile &t, uint32_t lds) {
    constexpr int FM = C::FM, FN = C::FN, S = C::NSTAGE;
    static_assert(FN == 2 && FM >= 2, "two products in turn; fragments one row of tiles ahead");
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
    xl.init(t.x, (uint32_t)a.ld, t.rows, t.len);
    wl.init(t.w, (uint32_t)a.ld, t.cols, t.len);
    const uint32_t chunk = xl.lane_chunk(), x_row = xl.lane_row((uint32_t)a.ld);
    const uint32_t w_row = C::BM == C::BN ? x_row : wl.lane_row((uint32_t)a.ld);
    constexpr int L = C::LOADS, XL = BlkLoader<C, C::BM>::IPW;
    const uint32_t frag = frag_lane();
    // This wave's scales of a K-block: those of 64 rows of X, or of 64 rows of W where each has its own; else the last
    // wave brings those of the tile's 128-row blocks of W, and the others none (zeros land in their places).
    const bool x_scales = wave < C::BM / 64, w_scales = WROWS ? wave * 256 >= C::SC_W : wave == C::NW - 1;
    const int sc_row = x_scales ? wave * 64 : WROWS ? wave * 64 - C::SC_W / 4 : 0;
    const float *sc_src = x_scales ? t.xs + sc_row : t.ws + sc_row;
    const int64_t sc_ld = x_scales ? a.xs_ld : WROWS ? a.ws_ld : 1;
    const int blocks = (t.cols + kBlk - 1) / kBlk;
    const uint32_t sc_bytes =
        x_scales   ? (uint32_t)max(t.rows - sc_row, 0) * 4u
        : w_scales ? WROWS ? (uint32_t)max(t.cols - sc_row, 0) * 4u : (uint32_t)((blocks - 1) * (int)a.ws_ld + 1) * 4u
                   : 0u;
    const uint32_t sc_lane = x_scales || WROWS ? 4u : 4u * (uint32_t)a.ws_ld;   // bytes from a lane's scale to the next

    // Ring positions by counters: the compiler would otherwise keep an address register for each read.
    auto stage = [&](int kt) { return lds + (uint32_t)((kt % S) * C::STAGE_BYTES); };
    auto scales = [&](int kt) { return lds + (uint32_t)(C::SC_OFF + (kt % (S + 1)) * C::SC_BYTES); };
    auto issue = [&](int i, int kt, uint32_t st, uint32_t sc) {   // load i of block kt
        if (i == 0)
            load_lds4(make_rsrc(sc_src + (int64_t)kt * sc_ld, kt < nk ? sc_bytes : 0u), (uint32_t)lane * sc_lane, 0,
                      sc + (uint32_t)wave * 256u);
        else if (i <= XL)
            xl.issue(i - 1, kt, st, x_row, chunk);
        else
            wl.issue(i - 1 - XL, kt, st + C::X_BYTES, w_row, chunk);
    };
    // Loads of block kt that go out with tile `at` after the barrier that frees its buffer: PER_TILE each, so that
    // the waves do not queue for the load path when they all leave the barrier.
    auto issue_with = [&](int at, int kt, uint32_t st, uint32_t sc) {
#pragma unroll
        for (int i = 0; i < L; ++i)
            if (i / C::PER_TILE == at) issue(i, kt, st, sc);
    };
    typedef __attribute__((address_space(3))) float lds_f32;
    const uint32_t x_rows = (uint32_t)(wm * C::WM * kBlk), w_rows = (uint32_t)(wn * 64 * kBlk);
    const uint32_t sw_at = (uint32_t)((C::NW - 1) * 256 + min(wn * 64 / kBlk, blocks - 1) * 4);
    BlkFrag w[FN], x[2];
    float sx[FM], sw = 1.0f;
    auto read_sx = [&](uint32_t sc) {
        if constexpr (!WROWS) sw = *(const lds_f32 *)(uintptr_t)(sc + sw_at);
        const uint32_t b = sc + (uint32_t)(wm * C::WM + (lane & 31)) * 4u;
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) sx[fm] = *((const lds_f32 *)(uintptr_t)b + fm * 32);
    };
    f32x16_t p[FN];   // the last one, zero at first, is added a step after the K-block it belongs to
    // Scales of W rows: lane k of each 16 holds that of the k-th of the lane half's 16 columns of a block tile, and a
    // multiplication takes it from there for all 16 lanes (row_newbcast); 16 registers of broadcast copies would cost
    // as much LDS time as the fragments.
    float sw_rows[FN] = {}, last = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) p[FN - 1][r] = 0.0f;
    auto join = [&](int fm, int fn) {   // p[fn] into its accumulator; last: the row's scale (times the tile's)
        asm volatile("" : "+v"(sw_rows[fn]));   // broadcast anew for each tile: kept, the copies would spill
        scaled_add<WROWS>(acc[fm][fn], p[fn], last, sw_rows[fn], std::make_integer_sequence<int, 16>{});
        asm volatile("" : "+v"(acc[fm][fn]));   // here, not past the next barrier
    };
    auto read_sw = [&](uint32_t sc) {
        if constexpr (WROWS) {
            const uint32_t b =
                sc + (uint32_t)(C::SC_W + (wn * 64 + ((lane & 15) >> 2) * 8 + (lane >> 5) * 4 + (lane & 3)) * 4);
#pragma unroll
            for (int fn = 0; fn < FN; ++fn) sw_rows[fn] = *((const lds_f32 *)(uintptr_t)b + fn * 32);
        }
    };
    // K-block kt
    auto block = [&](int kt) {
        uint32_t st = stage(kt), st1 = stage(kt + 1), sc = scales(kt), sc1 = scales(kt + 1);
        uint32_t stp = stage(kt + S - 1), scp = scales(kt + S - 1), scn = scales(kt + S);
        asm volatile("" : "+s"(st), "+s"(st1), "+s"(sc), "+s"(sc1), "+s"(stp), "+s"(scp), "+s"(scn));
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            if (fm == FM - 1) {
                wait_lgkm0();   // the block's last fragments are in registers
                if constexpr (C::EARLY_W) wait_vmcnt<L - 1 - XL>();
                else wait_vmcnt<(S - 2) * L>();
                lds_barrier();
            }
            if (C::EARLY_W && fm == 1) {
                wait_lgkm0();   // W of block kt is in every wave's registers behind this barrier
                lds_barrier();
            }
            const float s = sx[fm] * sw;
#pragma unroll
            for (int fn = 0; fn < FN; ++fn) {
                __builtin_amdgcn_sched_barrier(0);
                if (fn == 0) {
                    if (fm == 0) x[1] = read_frag<1 * 32 * kBlk>(st + x_rows + frag);
                    if (fm == 1 && FM > 2) x[0] = read_frag<2 * 32 * kBlk>(st + x_rows + frag);
                    if (fm == 2) x[1] = read_frag<3 * 32 * kBlk>(st + x_rows + frag);
                    if (fm == FM - 1) x[0] = read_frag<0>(st1 + x_rows + frag);
                }
                p[fn] = blk_product<F32>(w[fn], x[fm & 1]);
                __builtin_amdgcn_sched_barrier(0);
                if (fm == FM - 1)
                    w[fn] = fn == 0 ? read_frag<C::X_BYTES>(st1 + w_rows + frag)
                                    : read_frag<C::X_BYTES + 32 * kBlk>(st1 + w_rows + frag);
                if constexpr (C::EARLY_W) {
#pragma unroll
                    for (int i = 0; i < L; ++i)
                        if (i <= XL ? fm == FM - 1 && fn == i / 3 : fm == 1 + (i - 1 - XL) / 4 && fn == (i - 1 - XL) / 2 % 2)
                            issue(i, kt + S, st, scn);
                } else if (fm == FM - 1) {
                    issue_with(fn, kt + S, st, scn);
                } else {
                    issue_with(FN + fm * FN + fn, kt + S - 1, stp, scp);
                }
                if (fn > 0) join(fm, fn - 1);
                else join((fm + FM - 1) % FM, FN - 1);
                if (fm == 0 && fn == 0) read_sw(sc);
                last = s;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        read_sx(sc1);
    };
    // as if block -1 had come before
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
#pragma unroll
        for (int at = 0; at < FM * FN; ++at) issue_with(at, i, stage(i), scales(i));
    constexpr int EARLY = C::EARLY_W || 2 * C::PER_TILE >= L ? L : 2 * C::PER_TILE;
#pragma unroll
    for (int i = 0; i < EARLY; ++i) issue(i, S - 1, stage(S - 1), scales(S - 1));
    static_assert((L + C::PER_TILE - 1) / C::PER_TILE <= FM * FN, "a block's loads go out before the next barrier");
    wait_vmcnt<(S - 2) * L + EARLY>();
    lds_barrier();
    read_sx(scales(0));
    x[0] = read_frag<0>(stage(0) + x_rows + frag);
    w[0] = read_frag<C::X_BYTES>(stage(0) + w_rows + frag);
    w[1] = read_frag<C::X_BYTES + 32 * kBlk>(stage(0) + w_rows + frag);
    for (int kt = 0; kt < nk; ++kt) block(kt);
    join(FM - 1, FN - 1);
    wait_vmcnt<0>();   // the loads of blocks past the last, which write zeros
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
    t.x = a.x + (int64_t)m0 * a.ld + r0;
    t.w = a.w + (int64_t)n0 * a.ld + r0;
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
    a.ld = p.K;
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
    a.ld = (int)p.M;
    hipError_t e;
    if (p.f32) e = launch_wgrad<CfgM, true>(a, st);
    else e = p.bm == CfgM::BM ? launch_wgrad<CfgM, false>(a, st) : launch_wgrad<CfgL, false>(a, st);
    return check_hip(e, "mok_fp8_wgrad");
}

}  // namespace mok
