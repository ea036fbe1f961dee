// Products on operands in blocks of 128 (fp8_gemm.h): rows by weights, dense or
// grouped by expert, and the weight gradients.
#include <atomic>

#include "fp8_plan.h"
#include "fp8_tiles.h"

namespace mok {
namespace {

using CfgL = BlkCfg<256, 256, 2, 4, 2, 3, true>;
using CfgM = BlkCfg<128, 256, 2, 4, 3, 3>;

// One tile: output rows [m0, m0 + rows) x columns [n0, ..), contraction [k0, k0 + len).
struct BlkTile {
    const uint8_t *x, *w;    // first row at k0
    const float *xs, *ws;    // scales of the first row (W by tiles: the first block row) at k0
    int rows, cols, len;
    int64_t out;             // first element in out (and in a run's partials)
    bool refused;            // the result is NaN (CUT, see blk_tile)
    float *part;             // partials of the tile's run of the contraction
};

// ----------------------------------------------------------------------------- tiles

// Workgroup b of a segment of 8 * per workgroups -> tile; each XCD walks a contiguous range.
__device__ __forceinline__ int xcd_tile(int b, int per) { return (b % kXcds) * per + b / kXcds; }
// Tile id of total x cols in groups of kGroupM row tiles x all columns -> (row tile, column).
__device__ __forceinline__ void group_tile(int id, int total, int cols, int &mt, int &col) {
    const int gsize = kGroupM * cols, first = id / gsize * kGroupM, gm = min(kGroupM, total - first), r = id % gsize;
    mt = first + r % gm;
    col = r / gm;
}

struct RowTile {
    int e, m0, rows, nt, s;   // s: run of the contraction
};
// Workgroup b of tiles of bm rows, every one cut into `splits` runs; false: none.
__device__ __forceinline__ bool locate(const BlkArgs &a, int bm, int n_tiles, int splits, int b, RowTile &t) {
    const auto tiles = [bm](int n) { return (n + bm - 1) / bm; };
    const int total = count_tiles(a, tiles), cols = n_tiles * splits, all = total * cols;
    const int per = (all + kXcds - 1) / kXcds, id = xcd_tile(b, per);
    if (b / kXcds >= per || id >= all) return false;
    int mt, col;
    group_tile(id, total, cols, mt, col);
    t.nt = col % n_tiles;
    t.s = col / n_tiles;
    const Found f = find_tile(a, mt, tiles);
    t.e = f.e;
    t.m0 = f.lo + f.i * bm;
    t.rows = min(bm, f.n - f.i * bm);
    return true;
}

// Workgroup b of tiles of 256 rows and of 128 (half), which take 0.6 of their time:
// an expert's last rows go to a half tile if they fit, and where the whole tiles
// end in a round of at most kUnits / 2, that round takes them as halves (16,384 rows of
// 4 experts x 4,096 x 7,168: 459 -> 442 us). false: none.
constexpr int kUnits = 256;   // compute units
__device__ __forceinline__ bool locate_mixed(const BlkArgs &a, int n_tiles, int b, RowTile &t, bool &half) {
    const auto whole = [](int n) { return n / 256 + (n % 256 > 128); };
    const auto rest = [](int n) { return n % 256 > 0 && n % 256 <= 128 ? 1 : 0; };
    const int wholes = count_tiles(a, whole), rests = count_tiles(a, rest);
    int full = wholes * n_tiles, halves = full % kUnits;
    if (halves <= kUnits / 2) full -= halves;
    else halves = 0;
    const int all[3] = {full, 2 * halves, rests * n_tiles};
    int seg = 0, id = 0;
    for (; seg < 3; ++seg) {
        const int per = (all[seg] + kXcds - 1) / kXcds;
        id = xcd_tile(b, per);
        if (b < per * kXcds) break;
        b -= per * kXcds;
    }
    if (seg == 3 || id >= all[seg]) return false;
    t.s = 0;
    half = seg > 0;
    int mt;
    if (seg == 2) {
        group_tile(id, rests, n_tiles, mt, t.nt);
        const Found f = find_tile(a, mt, rest);
        t.e = f.e;
        t.m0 = f.lo + f.n / 256 * 256;
        t.rows = f.n % 256;
        return true;
    }
    group_tile(seg == 0 ? id : full + id / 2, wholes, n_tiles, mt, t.nt);
    const Found f = find_tile(a, mt, whole);
    const int below = f.i * 256 + (half ? id % 2 * 128 : 0);
    t.e = f.e;
    t.m0 = f.lo + below;
    t.rows = min(half ? 128 : 256, f.n - below);
    return true;
}

// ----------------------------------------------------------------------------- the tile's product

typedef uint32_t u32x4s_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void put16(uint32_t a, f32x4_t v) {
    *reinterpret_cast<__attribute__((address_space(3))) f32x4_t *>((uintptr_t)a) = v;
}
__device__ __forceinline__ f32x4_t get16(uint32_t a) {
    return *reinterpret_cast<const __attribute__((address_space(3))) f32x4_t *>((uintptr_t)a);
}

// out = addend + acc for the wave's 64 columns of a tile, N columns a row, rounded
// once. 32 rows at a time pass through the wave's own part of the LDS (whose
// accesses complete in order), so that stores and the addend's loads take whole
// runs of a row: a lane's accumulators hold 4 columns of one row. Staged as fp32
// rows of 256 bytes where an addend has to be added first, else as they are stored.
// 16-byte unit u of row r lies at u ^ (r % 16), in bf16 rows at u ^ (r / 2 % 8).
template <class C, bool F32>
__device__ __forceinline__ void store_tile(const f32x16_t (&acc)[C::FM][C::FN], const BlkTile &t, int N, void *out,
                                           const void *addend, uint32_t lds, int wm, int wn) {
    constexpr int FM = C::FM, FN = C::FN;
    static_assert(C::NW * 8192 <= C::LDS_BYTES, "8 KiB a wave");
    const int c0 = wn * 64, el = epi_lane(), row = el & 31, half = el >> 5;
    const int valid = min(t.cols - c0, 64);   // a multiple of 16
    constexpr uint32_t es = F32 ? 4u : 2u;
    const uint32_t row_bytes = (uint32_t)N * es;
    const uint32_t bytes = valid > 0 ? (uint32_t)(t.rows - 1) * row_bytes + (uint32_t)valid * es : 0u;
    const int64_t at_byte = (valid > 0 ? t.out + c0 : 0) * es;
    const brsrc_t dst = rows_rsrc(static_cast<char *>(out) + at_byte, bytes);
    const uint32_t area = lds + (uint32_t)wave_id() * 8192u;
    if (F32 || addend) {
        const brsrc_t add = rows_rsrc(addend ? static_cast<const char *>(addend) + at_byte : static_cast<char *>(out),
                                      addend ? bytes : 0u);
        const int pr = el >> 4, pu = el & 15;   // a pass: 4 rows of 16 lanes, 4 columns each
        const uint32_t v0 =
            pu * 4 < valid ? (uint32_t)(wm * C::WM + pr) * row_bytes + (uint32_t)pu * 4u * es : kOutOfRange;
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int g4 = 0; g4 < 4; ++g4) {
                    const uint32_t u = (uint32_t)(fn * 8 + g4 * 2 + half);
                    const f32x16_t &c = acc[fm][fn];
                    put16(area + (uint32_t)row * 256u + ((u ^ (uint32_t)(row & 15)) << 4),
                          f32x4_t{c[g4 * 4], c[g4 * 4 + 1], c[g4 * 4 + 2], c[g4 * 4 + 3]});
                }
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const int r = p * 4 + pr;
                const uint32_t v = v0 + (uint32_t)(fm * 32 + p * 4) * row_bytes;
                f32x4_t y = get16(area + (uint32_t)r * 256u + (uint32_t)((pu ^ (r & 15)) << 4));
                if constexpr (F32) {
                    if (addend) {
                        const u32x4s_t b = __builtin_amdgcn_raw_buffer_load_b128(add, (int)v, 0, 0);
#pragma unroll
                        for (int j = 0; j < 4; ++j) y[j] += __uint_as_float(b[j]);
                    }
                    const u32x4s_t w = {__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                                        __float_as_uint(y[3])};
                    __builtin_amdgcn_raw_buffer_store_b128(w, dst, (int)v, 0, 0);
                } else {
                    const uint2 b = bload8(add, v, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] += bf16_at(b, j);
                    bstore8_nt(dst, v, 0, make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])));
                }
            }
        }
    } else {
        const int pr = el >> 3, pu = el & 7;    // a pass: 8 rows of 8 lanes, 8 columns each
        const uint32_t v0 = pu * 8 < valid ? (uint32_t)(wm * C::WM + pr) * row_bytes + (uint32_t)pu * 16u : kOutOfRange;
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int g4 = 0; g4 < 4; ++g4) {
                    const f32x16_t &c = acc[fm][fn];
                    const uint32_t u = (uint32_t)(fn * 4 + g4);
                    u32x2v_t w;
                    w.x = pack_bf16x2(c[g4 * 4], c[g4 * 4 + 1]);
                    w.y = pack_bf16x2(c[g4 * 4 + 2], c[g4 * 4 + 3]);
                    const uint32_t to = area + (uint32_t)row * 128u + ((u ^ (uint32_t)(row >> 1 & 7)) << 4);
                    *reinterpret_cast<__attribute__((address_space(3))) u32x2v_t *>(
                        (uintptr_t)(to + (uint32_t)half * 8u)) = w;
                }
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int r = p * 8 + pr;
                const f32x4_t y = get16(area + (uint32_t)r * 128u + (uint32_t)((pu ^ (r >> 1 & 7)) << 4));
                const u32x4s_t w = {__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                                    __float_as_uint(y[3])};
                __builtin_amdgcn_raw_buffer_store_b128(w, dst, (int)(v0 + (uint32_t)(fm * 32 + p * 8) * row_bytes), 0,
                                                       2);
            }
        }
    }
}

// x of lane R of the lane's row of 16
template <int R>
__device__ __forceinline__ float lane_of_16(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + R, 0xF, 0xF, true));
}

// acc += p * s, or with a scale per W row (register R's in lane R of 16)
// acc += p * (s * sw_R): that is a second vector instruction for every value, which
// then take as long as the matrix cores. The products of scales come eight at a
// time, ahead of the additions that use them: one at a time, in one register, each
// waits for the one before (16,384 x 4,096 x 7,168 of 4 experts: 488 against 469 us;
// 412 with one scale a row).
template <int R0, int... R>
__device__ __forceinline__ void row_scales(float (&m)[sizeof...(R)], float s, float sw,
                                           std::integer_sequence<int, R...>) {
    ((m[R] = s * lane_of_16<R0 + R>(sw)), ...);
}
template <bool WROWS, int R0 = 0>
__device__ __forceinline__ void scaled_add(f32x16_t &acc, const f32x16_t &p, float s, float sw) {
    if constexpr (WROWS) {
        constexpr int G = 8;
        float m[G];
        row_scales<R0>(m, s, sw, std::make_integer_sequence<int, G>{});
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = 0; r < G; ++r) acc[R0 + r] = __builtin_fmaf(p[R0 + r], m[r], acc[R0 + r]);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (R0 + G < 16) scaled_add<WROWS, R0 + G>(acc, p, s, sw);
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[r] = __builtin_fmaf(p[r], s, acc[r]);
    }
}

// WROWS: W has a scale per row and block (weight gradients), else per 128 rows and
// block. F32: fp32 results, whose products are exact (blk_product). CUT: the
// contraction ends inside a 16-byte chunk, as an expert's run of rows may; what
// lies behind it there belongs to no expert and may be NaN, so it is cleared in
// LDS; and a run that is refused gets its NaN here. By itself, because a branch in
// the loop costs 1 to 2% (16,384 x 4,096 x 7,168 of 4 experts: 484 -> 497 us), code
// behind the loop 12% by its registers.
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
template <class C, bool WROWS, bool F32, bool CUT = false>
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
        scaled_add<WROWS>(acc[fm][fn], p[fn], last, sw_rows[fn]);
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
    auto clear_last = [&] {
        wait_vmcnt<0>();
        clear_behind<C>(stage(nk - 1), t.len);
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
                        if (i <= XL ? fm == FM - 1 && fn == i / 3
                                    : fm == 1 + (i - 1 - XL) / 4 && fn == (i - 1 - XL) / 2 % 2)
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
        if (CUT && kt == nk - 3) clear_last();   // all its loads are out, the barrier before its first read is to come
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
    if (CUT && nk > 0 && nk <= 2) clear_last();
    lds_barrier();
    read_sx(scales(0));
    x[0] = read_frag<0>(stage(0) + x_rows + frag);
    w[0] = read_frag<C::X_BYTES>(stage(0) + w_rows + frag);
    w[1] = read_frag<C::X_BYTES + 32 * kBlk>(stage(0) + w_rows + frag);
    for (int kt = 0; kt < nk; ++kt) block(kt);
    join(FM - 1, FN - 1);
    wait_vmcnt<0>();   // the loads of blocks past the last, which write zeros
    lds_barrier();   // the waves' staging areas lie where blocks were
    if constexpr (CUT) {
        const float more = t.refused ? __builtin_nanf("") : 0.0f;
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[fm][fn][r] += more;
    }

    if (a.splits > 1)   // fp32 partials, joined by a second kernel
        store_tile<C, true>(acc, t, a.N, t.part, nullptr, lds, wm, wn);
    else
        store_tile<C, F32>(acc, t, a.N, a.out, a.addend, lds, wm, wn);
}

__device__ __forceinline__ BlkTile matmul_tile(const BlkArgs &a, const RowTile &r, int bn) {
    const int n0 = r.nt * bn, nb = (a.N + kBlk - 1) / kBlk, kb = (a.K + kBlk - 1) / kBlk, b0 = r.s * a.run;
    BlkTile t;
    t.x = a.x + (int64_t)r.m0 * a.K + b0 * kBlk;
    t.w = a.w + ((int64_t)r.e * a.N + n0) * a.K + b0 * kBlk;
    t.xs = a.xs + (int64_t)b0 * a.xs_ld + r.m0;
    t.ws = a.ws + ((int64_t)r.e * nb + n0 / kBlk) * kb + b0;
    t.rows = r.rows;
    t.cols = min(bn, a.N - n0);
    t.len = a.splits > 1 ? min(a.K - b0 * kBlk, a.run * kBlk) : a.K;
    t.out = (int64_t)r.m0 * a.N + n0;
    t.part = a.part + (int64_t)r.s * a.M * a.N;
    return t;
}
__device__ __forceinline__ uint32_t lds_base() {
    extern __shared__ __attribute__((aligned(1024))) char lds_raw[];
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds_raw;
}

template <class C, bool F32>
__global__ __launch_bounds__(C::NT, 2) void blk_matmul(BlkArgs a) {
    RowTile r;
    if (!locate(a, C::BM, (a.N + C::BN - 1) / C::BN, a.splits, (int)blockIdx.x, r)) return;
    blk_tile<C, false, F32>(a, matmul_tile(a, r, C::BN), lds_base());
}

__global__ __launch_bounds__(CfgL::NT, 2) void blk_matmul_mixed(BlkArgs a) {
    static_assert(CfgL::BN == CfgM::BN && CfgL::NT == CfgM::NT, "one grid for both");
    RowTile r;
    bool half;
    if (!locate_mixed(a, (a.N + CfgL::BN - 1) / CfgL::BN, (int)blockIdx.x, r, half) || r.rows <= 0) return;
    const BlkTile t = matmul_tile(a, r, CfgL::BN);
    if (half) blk_tile<CfgM, false, false>(a, t, lds_base());
    else blk_tile<CfgL, false, false>(a, t, lds_base());
}

// The expert with the i-th most rows (of equal ones the lower index first), so that the longest tiles start first and
// the short ones fill the end; past 64 experts, expert i.
__device__ __forceinline__ int nth_longest(const BlkArgs &a, int i) {
    if (a.E < 2 || a.E > 64) return i;
    const int lane = threadIdx.x & 63;
    const int n = lane < a.E ? clamp_row(a.offsets[lane + 1], a.K) - clamp_row(a.offsets[lane], a.K) : 0;
    int rank = 0;
    for (int e = 0; e < a.E; ++e) {
        const int m = __builtin_amdgcn_readlane(n, e);
        rank += m > n || (m == n && e < lane) ? 1 : 0;
    }
    return __builtin_ctzll(__ballot(lane < a.E && rank == i));   // ranks are a permutation of 0 .. E - 1
}

// Weight gradients: rows of `x` are those of dy (output rows), rows of `w` those of x (columns).
template <class C, bool F32>
__global__ __launch_bounds__(C::NT, 2) void blk_wgrad(BlkArgs a) {
    const int gx = (a.N + C::BN - 1) / C::BN, gy = (a.M + C::BM - 1) / C::BM, cols = gx * a.splits;
    const int per = (cols * gy + kXcds - 1) / kXcds;
    const int id = xcd_tile((int)blockIdx.x % (per * kXcds), per);
    if (id >= cols * gy) return;
    const int e = nth_longest(a, (int)blockIdx.x / (per * kXcds));
    int mt, col;
    group_tile(id, gy, cols, mt, col);
    const int m0 = mt * C::BM, n0 = col % gx * C::BN, s = col / gx;
    int r0 = 0, r1 = a.K;
    bool refused = false;
    if (a.E > 0) {
        const int lo = uniform_i(clamp_row(a.offsets[e], a.K)), hi = uniform_i(clamp_row(a.offsets[e + 1], a.K));
        r0 = lo & ~(kBlk - 1);
        r1 = lo < hi ? hi : r0;   // an expert without rows may lie where another's run ended, inside a block
        // Operands have one scale for a block's rows, whoever they belong to: no run begins inside one. Only the device
        // knows the offsets, so the answer to one that does is NaN.
        refused = r0 < lo && lo < hi;
    }
    if (a.splits > 1) {   // this expert's blocks in equal runs
        const int run = ((r1 - r0 + kBlk - 1) / kBlk + a.splits - 1) / a.splits * kBlk;
        r0 += s * run;   // past the expert's end: an empty run
        r1 = min(r1, r0 + run);
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
    t.part = a.part + (int64_t)s * max(a.E, 1) * a.M * a.N;
    t.refused = refused;
    if (uniform_i((t.len & 15) | (int)refused)) blk_tile<C, true, F32, true>(a, t, lds_base());
    else blk_tile<C, true, F32>(a, t, lds_base());
}

// out = addend + sum of the runs' partials, in ascending order, 4 values a thread; 8 loads are in flight before the
// first is added. Rows of no expert (products by weights) stay as they were.
template <bool F32>
__global__ __launch_bounds__(256) void blk_join(BlkArgs a, int64_t quads, int64_t stride, bool rows) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= quads) return;
    if (rows && a.E > 0) {
        const int m = (int)(i / (a.N / 4));
        if (m < a.offsets[0] || m >= a.offsets[a.E]) return;
    }
    f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int r0 = 0; r0 < a.splits; r0 += 8) {
        f32x4_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = *reinterpret_cast<const f32x4_t *>(a.part + min(r0 + j, a.splits - 1) * stride + i * 4);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (r0 + j < a.splits) s += v[j];
    }
    if constexpr (F32) {
        if (a.addend) s += static_cast<const f32x4_t *>(a.addend)[i];
        static_cast<f32x4_t *>(a.out)[i] = s;
    } else {
        if (a.addend) {
            const uint2 b = static_cast<const uint2 *>(a.addend)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += bf16_at(b, j);
        }
        static_cast<uint2 *>(a.out)[i] = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    }
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

// Row tiles of bm rows: at most one more for each expert that has rows.
int64_t most_row_tiles(const BlkArgs &a, int bm) { return ceil_div(a.M, bm) + (a.E > 0 ? std::min(a.E, a.M) : 0); }
unsigned rounded(int64_t workgroups) { return (unsigned)(ceil_div(workgroups, kXcds) * kXcds); }

template <class K>
hipError_t launch_tiles(K *kernel, const char *name, unsigned grid, int threads, size_t lds,
                        std::atomic<uint64_t> &done, const BlkArgs &a, hipStream_t st) {
    const hipError_t e = allow_lds(kernel, lds, done);
    if (e != hipSuccess) return e;
    KernelTimer tm(name, st);
    kernel<<<grid, threads, lds, st>>>(a);
    return hipGetLastError();
}

template <class C, bool F32>
hipError_t launch_matmul(const BlkArgs &a, hipStream_t st) {
    static std::atomic<uint64_t> done{0};
    const unsigned grid = rounded(most_row_tiles(a, C::BM) * ceil_div(a.N, C::BN) * a.splits);
    return launch_tiles(blk_matmul<C, F32>, "fp8_matmul", grid, C::NT, C::LDS_BYTES, done, a, st);
}

hipError_t launch_mixed(const BlkArgs &a, hipStream_t st) {
    static std::atomic<uint64_t> done{0};
    // kUnits / 2 whole tiles as halves take as many workgroups again; each of the three segments is rounded up
    const unsigned grid = rounded(most_row_tiles(a, 256) * ceil_div(a.N, CfgL::BN) + kUnits / 2) + 3 * kXcds;
    constexpr size_t lds = CfgL::LDS_BYTES > CfgM::LDS_BYTES ? CfgL::LDS_BYTES : CfgM::LDS_BYTES;
    return launch_tiles(blk_matmul_mixed, "fp8_matmul", grid, CfgL::NT, lds, done, a, st);
}

template <class C, bool F32>
hipError_t launch_wgrad(const BlkArgs &a, hipStream_t st) {
    static std::atomic<uint64_t> done{0};
    const unsigned grid =
        rounded(ceil_div(a.N, C::BN) * ceil_div(a.M, C::BM) * a.splits) * (unsigned)std::max(a.E, 1);
    return launch_tiles(blk_wgrad<C, F32>, "fp8_wgrad", grid, C::NT, C::LDS_BYTES, done, a, st);
}

hipError_t launch_join(const BlkArgs &a, bool f32, int64_t values, bool rows, hipStream_t st) {
    const unsigned grid = (unsigned)ceil_div(values / 4, 256);
    KernelTimer tm("fp8_join", st);
    if (f32) blk_join<true><<<grid, 256, 0, st>>>(a, values / 4, values, rows);
    else blk_join<false><<<grid, 256, 0, st>>>(a, values / 4, values, rows);
    return hipGetLastError();
}

}  // namespace

mok_status launch_fp8_matmul(const BlkPlan &p, void *workspace, const uint8_t *a_elems, const float *a_scales,
                             const uint8_t *b_elems, const float *b_scales, const int32_t *offsets, void *out,
                             hipStream_t st) {
    BlkArgs a{};
    a.xs_ld = p.M;
    a.ws_ld = (p.K + kBlk - 1) / kBlk;
    a.x = a_elems;
    a.w = b_elems;
    a.xs = a_scales;
    a.ws = b_scales;
    a.offsets = offsets;
    a.out = out;
    a.part = static_cast<float *>(workspace);
    a.M = (int)p.M;
    a.N = p.N;
    a.K = p.K;
    a.E = p.E;
    a.ld = p.K;
    a.splits = p.splits;
    a.run = p.run;
    hipError_t e;
    if (p.few) e = launch_blk_few(a, p.few, p.few_w, p.f32, st);
    else if (p.bm == 256) e = launch_mixed(a, st);
    else e = p.f32 ? launch_matmul<CfgM, true>(a, st) : launch_matmul<CfgM, false>(a, st);
    if (e == hipSuccess && p.splits > 1) e = launch_join(a, p.f32, p.M * p.N, true, st);
    return check_hip(e, "mok_fp8_matmul");
}

mok_status launch_fp8_wgrad(const BlkPlan &p, void *workspace, const uint8_t *dy_elems, const float *dy_scales,
                            const uint8_t *x_elems, const float *x_scales, const int32_t *offsets, const void *addend,
                            void *out, hipStream_t st) {
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
    a.part = static_cast<float *>(workspace);
    a.M = p.N;
    a.N = p.K;
    a.K = (int)p.M;
    a.E = p.E;
    a.ld = (int)p.M;
    a.splits = p.splits;
    hipError_t e;
    if (p.f32) e = launch_wgrad<CfgM, true>(a, st);
    else e = p.bm == 128 ? launch_wgrad<CfgM, false>(a, st) : launch_wgrad<CfgL, false>(a, st);
    if (e == hipSuccess && p.splits > 1)
        e = launch_join(a, p.f32, (int64_t)std::max(p.E, 1) * p.N * p.K, false, st);
    return check_hip(e, "mok_fp8_wgrad");
}

}  // namespace mok
