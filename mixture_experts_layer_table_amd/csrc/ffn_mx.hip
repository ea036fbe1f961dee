// Gated feed-forward block in MXFP8: the four products with a weight operand
// run on the block-scaled MFMA (gemm8.h), every operand quantized along its
// contraction axis, 32 values per E8M0 scale:
//   gate/up  x (given quantized) x W_gate^T | W_up^T
//   down     a (quantized from its fp32 value in the gate/up epilogue) x W_down^T
//   dA       dy (quantized here) x W_down
//   dX       dh (quantized from its fp32 value in the dA epilogue) x W_gate | W_up
// h, the outputs and the weight gradients are BF16, as in ffn.hip, whose
// formulas and split over the contraction axis this file shares.
//
// Measured: forward 2,048 x 7,168 x 2,048 115 to 119 us over several cards (1,520
// to 1,570 TFLOP/s; its gate/up product has 128 tiles of 256 rows for 256 compute
// units: 128-row tiles instead, 71 us on one card, where 256 rows cut in two took 62
// and their join 15), 16,384 rows 0.69 ms (2,100; 0.74 with an addend); backward
// 16,384 rows 1.88 to 1.92 ms, of which the BF16 weight gradients are half the flops.
// A 128-row tile takes 0.5 to 0.6 us a K-step where the 256-row one takes 0.8, so it
// pays where it saves a split or a round. Both wait for their operands (2,048 rows'
// gate/up: 68 us on the fastest card; 64 without the MFMAs, 49 without the loads, 68
// without the fragment reads).
#include "ffn_parts.h"
#include "gemm8.h"
#include "kernels.h"
#include "mx_block.h"

namespace mok {
namespace {

using CfgA = TileCfg<256, 256, 2, 4, 4>;
using CfgH = TileCfg<128, 256, 2, 4, 4>;   // half the rows: twice the tiles before a product has to be split
using CfgS = TileCfg<128, 256, 2, 4, 6>;   // BF16 weight gradients
constexpr int kK8 = 64;                    // fp8 values per row and stage
static_assert(Fp8Stage<CfgA>::BK8 == kK8 && Fp8Stage<CfgH>::BK8 == kK8, "one K-step for both tiles");

__device__ __forceinline__ const uint16_t *as_pairs(const uint8_t *p) { return reinterpret_cast<const uint16_t *>(p); }

// MXFP8 codes staged in a FragStage array: 8-byte unit u of row r holds 8
// consecutive columns, 4 from lane half 0 and 4 from lane half 1.
template <class FS>
__device__ __forceinline__ uint32_t code_off(int r, int u, int lane) {
    return FS::at(r, u) + (uint32_t)((lane >> 5) * 4);
}
__device__ __forceinline__ void put4(uint32_t a, uint32_t v) {
    *reinterpret_cast<__attribute__((address_space(3))) uint32_t *>((uintptr_t)a) = v;
}
__device__ __forceinline__ void bstore1(brsrc_t r, uint32_t voff, uint32_t v) {
    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)v, r, (int)voff, 0, 0);
}
__device__ __forceinline__ void bstore2(brsrc_t r, uint32_t voff, uint32_t v) {
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)v, r, (int)voff, 0, 0);
}

struct Ffn8Args {
    int T, H, I, n_tiles, splits, len;
    const uint8_t *x, *xs;                // the product's row operand and its scales
    const uint8_t *w0, *w0s, *w1, *w1s;   // its weights (w1: W_up where both are needed)
    const uint16_t *addend, *h_in;
    uint16_t *out, *h, *a, *dh;
    uint8_t *q, *qs;                      // what the epilogue quantizes: a, or dh
    float *part;
};

// Members that every problem below shares: loaders, tile and K-step issue.
template <class Cfg>
struct Ffn8Base {
    using C = Cfg;
    using S8 = Fp8Stage<C>;
    using Args = Ffn8Args;
    static constexpr size_t LDS = S8::LDS_BYTES;   // dynamic LDS of the launch
    RowLoader<C, C::BM> xl;
    RowLoader<C, C::BN> wl;
    ScaleLoader<C> sl;
    static constexpr int LOADS_PER_STAGE = RowLoader<C, C::BM>::IPW + RowLoader<C, C::BN>::IPW;
    FfnTile t;
    int nk;
    Args a;

    // false: no tile; k0: the run's first value of a contraction axis of K values
    template <bool TILED>
    __device__ bool begin(const Args &args, int b, int K, int &k0) {
        a = args;
        if (!ffn_tile(a.T, C::BM, a.n_tiles, a.splits, b, t)) return false;
        k0 = t.s * a.len * kK8;
        nk = min(a.len, K / kK8 - t.s * a.len);
        if constexpr (TILED) {
            const uint32_t off = tiled_at((uint32_t)a.T, (uint32_t)t.m0, (uint32_t)k0);
            xl.init_tiled(a.x + off, (uint32_t)a.T * 64u, (uint32_t)a.T * (uint32_t)K - off);
            __builtin_assume(xl.kblock != 0);
        } else {
            xl.init(as_pairs(a.x + (int64_t)t.m0 * K + k0), K / 2, t.rows);
        }
        return true;
    }
    __device__ const uint8_t *x_scales(int K, int k0) const { return a.xs + (int64_t)t.m0 * (K / 32) + k0 / 32; }
    __device__ void issue(int kt, uint32_t stage) {
        sl.issue(kt, stage - (uint32_t)((kt % C::NSTAGE) * S8::BYTES));   // chunk first: see ScaleLoader
        xl.issue(kt * C::BK, stage);
        wl.issue(kt * C::BK, stage + C::X_BYTES);
    }
    __device__ int wrow(int wn, int fn) const { return wn * C::WN + fn * 32; }
};

template <class Cfg>
struct FfnGateUp8 : Ffn8Base<Cfg> {
    using B = Ffn8Base<Cfg>;
    using typename B::Args;
    using typename B::C;
    using typename B::S8;
    using B::a;
    using B::sl;
    using B::t;
    using B::wl;
    using B::xl;
    using B::x_scales;
    __device__ bool setup(const Args &args, int b) {
        int k0;
        const int H = args.H;
        if (!B::template begin<false>(args, b, H, k0)) return false;
        const int i0 = t.nt * (C::BN / 2), nw = min(C::BN / 2, a.I - i0);
        const int64_t wo = (int64_t)i0 * H + k0, so = (int64_t)i0 * (H / 32) + k0 / 32;
        wl.init_split_rows(as_pairs(a.w0 + wo), as_pairs(a.w1 + wo), H / 2, nw);
        sl.init(x_scales(H, k0), t.rows, H / 32, a.w0s + so, nw, H / 32, a.w1s + so);
        return true;
    }
    // gate rows of the W tile pair with the up rows BN/2 further inside one wave
    __device__ int wrow(int wn, int fn) const {
        return fn < C::FN / 2 ? wn * (C::WN / 2) + fn * 32 : C::BN / 2 + wn * (C::WN / 2) + (fn - C::FN / 2) * 32;
    }
    __device__ void epilogue(f32x16_t (&acc)[C::FM][C::FN], int wm, int wn) {
        constexpr size_t END = S8::LDS_BYTES;
        const int I = a.I, ib0 = t.nt * (C::BN / 2) + wn * (C::WN / 2);
        const bool live = ib0 < I;   // I % 128 == 0: the wave's i are all valid or all past I
        if (a.splits > 1) {
            store_partials<C>(acc, a.part + ((int64_t)t.s * a.T + t.m0) * 2 * I, 2 * I, t.rows, wm, live, [&](int fn) {
                return fn < C::FN / 2 ? ib0 + fn * 32 : I + ib0 + (fn - C::FN / 2) * 32;
            });
            return;
        }
        if (!live) return;
        if (a.h) {
            const uint32_t h_row = 4u * (uint32_t)I;
            const uint32_t h_col =
                2u * (uint32_t)(ib0 + (FragStage<C, END>::pass_col(epi_lane()) >= C::WN / 2 ? I - C::WN / 2 : 0));
            staged_rows<C, END>([&](int fm, int fn, int g4, int j) { return acc[fm][fn][g4 * 4 + j]; },
                                rows_rsrc(a.h + (int64_t)t.m0 * 2 * I, (uint32_t)t.rows * h_row),
                                [&](int fm, int r) -> uint32_t {
                                    return (uint32_t)(wm * C::WM + fm * 32 + r) * h_row + h_col;
                                });
        }
        // a: codes of one 32-block of i per row, staged as rows of 32 bytes
        using FS = FragStage<C, END>;
        static_assert(C::FN == 2, "one gate and one up block of 32 columns per wave");
        const int lane = epi_lane();
        const uint32_t area = FS::area(wave_id(), 1);
        const brsrc_t qres = rows_rsrc(a.q, (uint32_t)a.T * (uint32_t)I);
        const uint32_t q0 = tiled_at((uint32_t)a.T, (uint32_t)t.m0, (uint32_t)(ib0 + (lane & 3) * 8));
        const brsrc_t sres = rows_rsrc(a.qs + (int64_t)t.m0 * (I / 32), (uint32_t)t.rows * (uint32_t)(I / 32));
#pragma unroll
        for (int fm = 0; fm < C::FM; ++fm) {
            const uint32_t m0 = (uint32_t)(wm * C::WM + fm * 32);
            Block16 av;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float hg = acc[fm][0][e], hu = acc[fm][1][e];
                av.v[e] = hg * sigmoidf_(hg) * hu;
            }
            const Enc16 q8 = encode_block16(av);
#pragma unroll
            for (int g4 = 0; g4 < 4; ++g4) put4(area + code_off<FS>(lane & 31, g4, lane), q8.enc[g4]);
#pragma unroll
            for (int p = 0; p < 2; ++p) {   // 16 rows a pass, 8 codes a lane
                const int r = p * 16 + (lane >> 2);
                const uint32_t m = m0 + (uint32_t)r;
                bstore8_nt(qres, m < (uint32_t)t.rows ? q0 + m * 64u : kOutOfRange, 0,
                           FS::get(area + FS::at(r, lane & 3)));
            }
            bstore1(sres, lane < 32 ? (m0 + (uint32_t)lane) * (uint32_t)(I / 32) + (uint32_t)(ib0 / 32) : kOutOfRange,
                    q8.scale);
        }
    }
};

template <class Cfg>
struct FfnDown8 : Ffn8Base<Cfg> {
    using B = Ffn8Base<Cfg>;
    using typename B::Args;
    using typename B::C;
    using typename B::S8;
    using B::a;
    using B::sl;
    using B::t;
    using B::wl;
    using B::xl;
    using B::x_scales;
    __device__ bool setup(const Args &args, int b) {
        int k0;
        const int I = args.I;
        if (!B::template begin<true>(args, b, I, k0)) return false;
        const int n0 = t.nt * C::BN, nw = min(C::BN, a.H - n0);
        wl.init(as_pairs(a.w0 + (int64_t)n0 * I + k0), I / 2, nw);
        sl.init(x_scales(I, k0), t.rows, I / 32, a.w0s + (int64_t)n0 * (I / 32) + k0 / 32, nw, I / 32);
        return true;
    }
    __device__ void epilogue(f32x16_t (&acc)[C::FM][C::FN], int wm, int wn) {
        dense_epilogue<C, S8::LDS_BYTES>(acc, t, a.T, a.H, a.splits, wm, wn, a.addend, a.out, a.part);
    }
};

template <class Cfg>
struct FfnDA8 : Ffn8Base<Cfg> {
    using B = Ffn8Base<Cfg>;
    using typename B::Args;
    using typename B::C;
    using typename B::S8;
    using B::a;
    using B::sl;
    using B::t;
    using B::wl;
    using B::xl;
    using B::x_scales;
    __device__ bool setup(const Args &args, int b) {
        int k0;
        const int H = args.H;
        if (!B::template begin<true>(args, b, H, k0)) return false;
        const int i0 = t.nt * C::BN, nw = min(C::BN, a.I - i0);
        wl.init(as_pairs(a.w0 + (int64_t)i0 * H + k0), H / 2, nw);
        sl.init(x_scales(H, k0), t.rows, H / 32, a.w0s + (int64_t)i0 * (H / 32) + k0 / 32, nw, H / 32);
        return true;
    }
    // four staged arrays of 4 KiB a wave, which may be more than the tile's own LDS
    static constexpr size_t LDS = S8::LDS_BYTES > 4 * (size_t)C::NW * 4096 ? S8::LDS_BYTES : 4 * (size_t)C::NW * 4096;
    // As the BF16 dA: h rows come in and dh and a rows leave as whole row runs,
    // staged one 32-row fragment at a time through row descriptors; dh's codes
    // take a fourth staging array, their scales one 2-byte store a row and half.
    // (At 16,384 x 7,168 x 2,048: 307 us; 411 with each lane's pieces stored
    // directly and quantized out of line, every call waiting for all stores in
    // flight. The tiles write and read 400 MB in two bursts, 78 us of HBM time.)
    __device__ void epilogue(f32x16_t (&acc)[C::FM][C::FN], int wm, int wn) {
        using FS = FragStage<C, LDS>;
        static_assert(C::FN == 2 && LDS >= 4 * (size_t)C::NW * FS::BYTES, "four staged arrays");
        const int I = a.I, ib0 = t.nt * C::BN + wn * C::WN;
        const bool live = ib0 < I;   // I % 128 == 0: a wave's 64 columns are all valid or none
        if (a.splits > 1) {
            store_partials<C>(acc, a.part + ((int64_t)t.s * a.T + t.m0) * I, I, t.rows, wm, live,
                              [&](int fn) { return ib0 + fn * 32; });
            return;
        }
        const int lane = epi_lane();
        const int ib = live ? ib0 : 0;
        const uint32_t rows = live ? (uint32_t)t.rows : 0u;
        const uint32_t sg = FS::area(wave_id(), 4), su = sg + FS::BYTES, sa = su + FS::BYTES, sq = sa + FS::BYTES;
        const uint32_t up = 2u * (uint32_t)I, row_bytes = 2u * up, sc_bytes = up / 32;
        const brsrc_t hres = rows_rsrc(a.h_in + (int64_t)t.m0 * 2 * I, rows * row_bytes);
        const brsrc_t dres = rows_rsrc(a.dh + (int64_t)t.m0 * 2 * I, rows * row_bytes);
        const brsrc_t ares = rows_rsrc(a.a + (int64_t)t.m0 * I, rows * up);
        const brsrc_t qres = rows_rsrc(a.q, (uint32_t)a.T * up);
        const brsrc_t sres = rows_rsrc(a.qs + (int64_t)t.m0 * sc_bytes, rows * sc_bytes);
        // the lane's byte offsets at pass 0 of fragment 0; pass p of fragment fm lies step(fm, p) rows further.
        // A row's 128 staged code bytes are 64 of the gate half and 64 of the up half: one block of each.
        const uint32_t row0 = (uint32_t)(wm * C::WM + FS::pass_row(0, lane));
        const uint32_t d0 = row0 * row_bytes + 2u * (uint32_t)(ib + FS::pass_col(lane));
        const uint32_t a0 = row0 * up + 2u * (uint32_t)(ib + FS::pass_col(lane));
        const uint32_t q0 = tiled_at((uint32_t)a.T, (uint32_t)t.m0 + row0,
                                     (uint32_t)(ib + (lane % 8) * 8 + (lane % 16 >= 8 ? I : 0)));
        auto step = [](int fm, int p) { return (uint32_t)(fm * 32 + p * FS::RPP); };
        uint2 hg[FS::PASSES], hu[FS::PASSES];
        auto load_h = [&](int fm) {
#pragma unroll
            for (int p = 0; p < FS::PASSES; ++p) {
                hg[p] = bload8(hres, d0 + step(fm, p) * row_bytes, 0);
                hu[p] = bload8(hres, d0 + step(fm, p) * row_bytes, up);
            }
        };
        load_h(0);
#pragma unroll
        for (int fm = 0; fm < C::FM; ++fm) {
            // LDS offsets are worked out anew for each fragment: kept across all
            // four they spill, and a reload waits behind every store in flight
            const int lane = epi_lane();
#pragma unroll
            for (int p = 0; p < FS::PASSES; ++p) {
                FS::put(sg + FS::pass_off(p, lane), hg[p]);
                FS::put(su + FS::pass_off(p, lane), hu[p]);
            }
            __builtin_amdgcn_sched_barrier(0);   // phases stay in order: keeps live ranges short
            uint32_t sc = 0;   // lanes below 32: the gate half's two scale bytes of row lane, the others: the up half's
#pragma unroll
            for (int fn = 0; fn < C::FN; ++fn) {
                Block16 dg, du;
#pragma unroll
                for (int g4 = 0; g4 < 4; ++g4) {
                    const uint32_t o = FS::frag_off(fn, g4, lane);
                    const int e = g4 * 4;
                    const uint2 hg2 = FS::get(sg + o), hu2 = FS::get(su + o);
                    float av[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const GluGrad g = glu_backward(acc[fm][fn][e + j], bf16_at(hg2, j), bf16_at(hu2, j));
                        av[j] = g.a;
                        dg.v[e + j] = g.dg;
                        du.v[e + j] = g.du;
                    }
                    FS::put(sg + o, pack4(dg.v[e], dg.v[e + 1], dg.v[e + 2], dg.v[e + 3]));
                    FS::put(su + o, pack4(du.v[e], du.v[e + 1], du.v[e + 2], du.v[e + 3]));
                    FS::put(sa + o, pack4(av[0], av[1], av[2], av[3]));
                }
                const Enc16 qg = encode_block16(dg), qu = encode_block16(du);
#pragma unroll
                for (int g4 = 0; g4 < 4; ++g4) {
                    put4(sq + code_off<FS>(lane & 31, fn * 4 + g4, lane), qg.enc[g4]);
                    put4(sq + code_off<FS>(lane & 31, 8 + fn * 4 + g4, lane), qu.enc[g4]);
                }
                sc |= (lane < 32 ? qg.scale : qu.scale) << (8 * fn);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (fm + 1 < C::FM) load_h(fm + 1);   // in flight while this fragment's rows are stored
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int p = 0; p < FS::PASSES; ++p) {
                const uint32_t o = FS::pass_off(p, lane), v = d0 + step(fm, p) * row_bytes;
                bstore8_nt(dres, v, 0, FS::get(sg + o));
                bstore8_nt(dres, v, up, FS::get(su + o));
                bstore8_nt(ares, a0 + step(fm, p) * up, 0, FS::get(sa + o));
                bstore8_nt(qres, row0 + step(fm, p) < rows ? q0 + step(fm, p) * 64u : kOutOfRange, 0, FS::get(sq + o));
            }
            const uint32_t sr = (uint32_t)(wm * C::WM + fm * 32 + (lane & 31)) * sc_bytes;
            bstore2(sres, sr + (uint32_t)((ib + (lane < 32 ? 0 : I)) / 32), sc);
        }
    }
};

template <class Cfg>
struct FfnDX8 : Ffn8Base<Cfg> {
    using B = Ffn8Base<Cfg>;
    using typename B::Args;
    using typename B::C;
    using typename B::S8;
    using B::a;
    using B::sl;
    using B::t;
    using B::wl;
    using B::xl;
    using B::x_scales;
    __device__ bool setup(const Args &args, int b) {
        int k0;
        const int I = args.I;
        if (!B::template begin<true>(args, b, 2 * I, k0)) return false;
        const int n0 = t.nt * C::BN, nw = min(C::BN, a.H - n0);
        const int64_t wo = (int64_t)n0 * I, so = (int64_t)n0 * (I / 32);
        const uint8_t *xs = x_scales(2 * I, k0);
        if (k0 < I) {   // the run starts among the gate columns and may go on into the up columns
            wl.init(as_pairs(a.w0 + wo + k0), I / 2, nw, as_pairs(a.w1 + wo), (I - k0) / 2);
            sl.init(xs, t.rows, 2 * I / 32, a.w0s + so + k0 / 32, nw, I / 32, nullptr, a.w1s + so, I - k0);
        } else {
            wl.init(as_pairs(a.w1 + wo + (k0 - I)), I / 2, nw);
            sl.init(xs, t.rows, 2 * I / 32, a.w1s + so + (k0 - I) / 32, nw, I / 32);
        }
        return true;
    }
    __device__ void epilogue(f32x16_t (&acc)[C::FM][C::FN], int wm, int wn) {
        dense_epilogue<C, S8::LDS_BYTES>(acc, t, a.T, a.H, a.splits, wm, wn, a.addend, a.out, a.part);
    }
};

// dy along H: a thread takes 8 values, 4 neighbouring lanes one 32-block; a
// workgroup 4 rows of 512 columns, whose blocks' rows lie side by side.
constexpr int kQRows = 4, kQCols = 512;
__global__ __launch_bounds__(64 * kQRows) void ffn_quantize_rows(const uint16_t *__restrict__ src, int T, int H,
                                                                 uint8_t *__restrict__ el, uint8_t *__restrict__ sc) {
    const uint32_t chunks = (uint32_t)(H + kQCols - 1) / kQCols;
    const int t = (int)(blockIdx.x / chunks) * kQRows + (int)(threadIdx.x >> 6);
    const int k = (int)(blockIdx.x % chunks) * kQCols + (int)(threadIdx.x & 63) * 8;
    if (t >= T || k >= H) return;   // whole groups of 4 lanes: rows are multiples of 128 values
    const uint4 x = *reinterpret_cast<const uint4 *>(src + (int64_t)t * H + k);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = max(amax, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
    const uint32_t sb = mx_scale_byte_bf16(amax);
    const int e = (int)sb - 127;
    const uint32_t nan = mx_nan_bf16(amax);
    *reinterpret_cast<uint2 *>(el + tiled_at((uint32_t)T, (uint32_t)t, (uint32_t)k)) =
        make_uint2(e4m3x4_bf16(w[0], w[1], e, nan), e4m3x4_bf16(w[2], w[3], e, nan));
    if (k % 32 == 0) sc[((int64_t)t * H + k) / 32] = (uint8_t)sb;
}

template <class P>
__global__ __launch_bounds__(P::C::NT, 2) void ffn_gemm8(Ffn8Args args) {
    extern __shared__ __attribute__((aligned(1024))) char lds_raw[];
    P p;
    if (!p.setup(args, (int)blockIdx.x)) return;
    gemm8_tile(p, (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds_raw);
}

// dW_gate | dW_up and dW_down (BF16 tiles), then dx (block-scaled tiles), in one launch.
template <class PX, class PW>
__global__ __launch_bounds__(PX::C::NT, 2) void ffn_grads8(FfnWgradArgs gu, FfnWgradArgs wd, Ffn8Args ax, int g0,
                                                           int g1) {
    extern __shared__ __attribute__((aligned(1024))) char lds_raw[];
    const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds_raw;
    int b = (int)blockIdx.x;
    if (b < g0 + g1) {
        PW p;
        if (!p.setup(b < g0 ? gu : wd, b < g0 ? b : b - g0)) return;
        gemm_tile(p, lds);
    } else {
        PX p;
        if (!p.setup(ax, b - g0 - g1)) return;
        gemm8_tile(p, lds);
    }
}

template <class P>
hipError_t launch_product8(const char *name, unsigned grid, const Ffn8Args &a, hipStream_t st) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds(ffn_gemm8<P>, P::LDS, done);
    if (e != hipSuccess) return e;
    KernelTimer tm(name, st);
    ffn_gemm8<P><<<grid, P::C::NT, P::LDS, st>>>(a);
    return hipGetLastError();
}

template <template <class> class P>
hipError_t product8(const char *name, const FfnSplit &s, Ffn8Args a, int n_tiles, hipStream_t st) {
    a.n_tiles = n_tiles;
    a.splits = s.splits;
    a.len = s.len;
    const unsigned grid = ffn_grid(a.T, s.bm, n_tiles, s.splits);
    return s.bm == CfgH::BM ? launch_product8<P<CfgH>>(name, grid, a, st) : launch_product8<P<CfgA>>(name, grid, a, st);
}

template <class CX, class CW>
hipError_t launch_grads8(const FfnWgradArgs &gu, const FfnWgradArgs &wd, const Ffn8Args &ax, hipStream_t st) {
    using PX = FfnDX8<CX>;
    static std::atomic<uint64_t> done{0};
    auto *k = ffn_grads8<PX, FfnWgrad<CW>>;
    constexpr size_t lds = PX::LDS > CW::LDS_BYTES ? PX::LDS : CW::LDS_BYTES;
    const hipError_t e = allow_lds(k, lds, done);
    if (e != hipSuccess) return e;
    const unsigned g0 = wgrad_grid(gu.M, gu.N, CW::BM), g1 = wgrad_grid(wd.M, wd.N, CW::BM);
    const unsigned gx = ffn_grid(ax.T, CX::BM, ax.n_tiles, ax.splits);
    KernelTimer tm("ffn_grads_mx", st);
    k<<<g0 + g1 + gx, CX::NT, lds, st>>>(gu, wd, ax, (int)g0, (int)g1);
    return hipGetLastError();
}

}  // namespace

hipError_t ffn_mx_forward(const FfnPlan &p, char *ws, const uint8_t *x_elems, const uint8_t *x_scales,
                          const mok_weights &w, const uint16_t *addend, uint16_t *out, uint16_t *h, hipStream_t st) {
    Ffn8Args a{};
    a.T = (int)p.T;
    a.H = p.H;
    a.I = p.I;
    a.x = x_elems;
    a.xs = x_scales;
    a.w0 = w.gate_elems;
    a.w0s = w.gate_scales;
    a.w1 = w.up_elems;
    a.w1s = w.up_scales;
    a.h = h;
    a.q = reinterpret_cast<uint8_t *>(ws + p.a_q);
    a.qs = reinterpret_cast<uint8_t *>(ws + p.a_qs);
    a.part = reinterpret_cast<float *>(ws + p.part);
    hipError_t e = product8<FfnGateUp8>("ffn_gate_up_mx", p.gate_up, a, (int)ceil_div(p.I, kTileN / 2), st);
    if (e != hipSuccess) return e;
    if (p.gate_up.splits > 1) {
        KernelTimer tm("ffn_join_act", st);
        ffn_join_act<true><<<join_grid(p.T, p.I), 256, 0, st>>>(a.part, p.gate_up.splits, a.T, a.I, h, nullptr, a.q,
                                                                a.qs);
    }
    a.x = a.q;
    a.xs = a.qs;
    a.w0 = w.down_elems;
    a.w0s = w.down_scales;
    a.addend = addend;
    a.out = out;
    e = product8<FfnDown8>("ffn_down_mx", p.down, a, (int)ceil_div(p.H, kTileN), st);
    if (e == hipSuccess && p.down.splits > 1) {
        KernelTimer tm("ffn_join_out", st);
        ffn_join_out<<<join_grid(p.T, p.H), 256, 0, st>>>(a.part, p.down.splits, a.T, a.H, addend, out);
        e = hipGetLastError();
    }
    return e;
}

hipError_t ffn_mx_backward(const FfnPlan &p, char *ws, const uint16_t *x, const mok_weights &w, const uint16_t *h,
                           const uint16_t *dy, const uint16_t *addend, uint16_t *dx, uint16_t *dw_gate, uint16_t *dw_up,
                           uint16_t *dw_down, hipStream_t st) {
    Ffn8Args a{};
    a.T = (int)p.T;
    a.H = p.H;
    a.I = p.I;
    a.a = reinterpret_cast<uint16_t *>(ws + p.a);
    a.dh = reinterpret_cast<uint16_t *>(ws + p.dh);
    a.q = reinterpret_cast<uint8_t *>(ws + p.dh_q);
    a.qs = reinterpret_cast<uint8_t *>(ws + p.dh_qs);
    a.part = reinterpret_cast<float *>(ws + p.part);
    hipError_t e = hipSuccess;
    if (p.T > 0) {
        uint8_t *dyq = reinterpret_cast<uint8_t *>(ws + p.dy_q), *dyqs = reinterpret_cast<uint8_t *>(ws + p.dy_qs);
        {
            const unsigned grid = (unsigned)(ceil_div(p.T, kQRows) * ceil_div(p.H, kQCols));
            KernelTimer tm("ffn_quantize_rows", st);
            ffn_quantize_rows<<<grid, 64 * kQRows, 0, st>>>(dy, a.T, p.H, dyq, dyqs);
        }
        a.x = dyq;
        a.xs = dyqs;
        a.w0 = w.down_elems;
        a.w0s = w.down_scales;
        a.h_in = h;
        e = product8<FfnDA8>("ffn_da_mx", p.da, a, (int)ceil_div(p.I, kTileN), st);
        if (e != hipSuccess) return e;
        if (p.da.splits > 1) {
            KernelTimer tm("ffn_join_da", st);
            ffn_join_da<true><<<join_grid(p.T, p.I), 256, 0, st>>>(a.part, p.da.splits, a.T, a.I, h, a.dh, a.a, a.q,
                                                                   a.qs);
        }
    }
    a.x = a.q;
    a.xs = a.qs;
    a.w0 = w.gate_elems;
    a.w0s = w.gate_scales;
    a.w1 = w.up_elems;
    a.w1s = w.up_scales;
    a.addend = addend;
    a.out = dx;
    a.n_tiles = (int)ceil_div(p.H, kTileN);
    a.splits = p.dx.splits;
    a.len = p.dx.len;
    const FfnWgradArgs gu{a.T, p.H, 2 * p.I, p.I, p.I, x, a.dh, dw_gate, dw_up};
    const FfnWgradArgs wd{a.T, p.I, p.H, p.H, p.H, a.a, dy, dw_down, nullptr};
    const bool small_w = p.wgrad_bm == CfgS::BM;
    if (p.dx.bm == CfgH::BM)
        e = small_w ? launch_grads8<CfgH, CfgS>(gu, wd, a, st) : launch_grads8<CfgH, CfgA>(gu, wd, a, st);
    else
        e = small_w ? launch_grads8<CfgA, CfgS>(gu, wd, a, st) : launch_grads8<CfgA, CfgA>(gu, wd, a, st);
    if (e == hipSuccess && p.T > 0 && p.dx.splits > 1) {
        KernelTimer tm("ffn_join_out", st);
        ffn_join_out<<<join_grid(p.T, p.H), 256, 0, st>>>(a.part, p.dx.splits, a.T, a.H, addend, dx);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace mok
