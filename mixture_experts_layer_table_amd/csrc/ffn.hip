// Gated feed-forward block in BF16, forward and backward: the dense (always
// taken) expert that runs beside the routed ones.
//   h = x [W_gate | W_up],  a = silu(h_g) * h_u,  out = addend + a W_down
//   G = dy W_down^T,  dh_u = G silu(h_g),  dh_g = G h_u s (1 + h_g (1 - s)), s = sigmoid(h_g)
//   dx = addend + dh_g W_gate^T + dh_u W_up^T
//   dW_gate | dW_up = x^T [dh_g | dh_u],  dW_down = a^T dy
// Both projections, the activation and their product are one kernel: a tile
// holds matching gate and up columns, and its epilogue writes a (and the saved
// h). The tiles are the library's BF16 tile engine (gemm.h).
//
// A few rows (ffn_few.hip) take kernels of their own. Somewhat more still leave
// most compute units without a tile, so a product is then cut along its
// contraction axis (ffn_plan.cpp) and its fp32 partials are added by a second,
// elementwise kernel that also does the epilogue's work. The weight gradients
// and dx all wait for dh alone and run as one launch, whose tiles fill each
// other's tails.
//
// Bound by the matrix cores and their operand loads together (the tile engine)
// where there are many rows: forward 16,384 x 7,168 x 2,048 1.12 ms, 1,290
// TFLOP/s (8,192^3 in the library's dense product with this weight layout:
// 1,240 - 1,280), backward 2.37 ms, 1,220. With few, by each kernel's fixed 5 us
// of launch and first loads: backward 1,001 x 4,096 x 1,024 79 us (630 TFLOP/s).
#include "ffn_few.h"
#include "ffn_parts.h"
#include "kernels.h"

namespace mok {
namespace {

using CfgA = TileCfg<256, 256, 2, 4, 4>;   // as the layer's: 4 stages of 32 KiB
using CfgS = TileCfg<128, 256, 2, 4, 6>;   // 6 stages of 24 KiB
// CfgS at half the LDS and at most 128 registers: two workgroups per compute
// unit, one's stores beside the other's loads
using CfgW = TileCfg<128, 256, 2, 4, 3, 4>;
static_assert(CfgA::BN == kTileN && CfgS::BN == kTileN && CfgW::BN == kTileN,
              "host sizing assumes kTileN-column tiles");

struct FfnArgs {
    int T, H, I, n_tiles, splits, len;
    const uint16_t *x;          // the product's row operand
    const uint16_t *w0, *w1;    // its weights (w1: W_up where both are needed)
    const uint16_t *addend, *h_in;
    uint16_t *out, *h, *a, *dh;
    float *part;
};

// a = silu(x W_gate) * (x W_up): both projections in one tile
template <class Cfg>
struct FfnGateUp {
    using C = Cfg;
    using Args = FfnArgs;
    static constexpr bool X_TRANS = false, W_TRANS = true;
    RowLoader<C, C::BM> xl;
    TransLoader<C, C::BN> wl;
    static constexpr int LOADS_PER_STAGE = RowLoader<C, C::BM>::IPW + TransLoader<C, C::BN>::IPW;
    FfnTile t;
    int i0, nk;
    Args a;
    __device__ int mvalid() const { return t.rows; }

    __device__ bool setup(const Args &args, int b) {
        a = args;
        if (!ffn_tile(a.T, C::BM, a.n_tiles, a.splits, b, t)) return false;
        i0 = t.nt * (C::BN / 2);
        const int k0 = t.s * a.len * C::BK;
        xl.init(a.x + (int64_t)t.m0 * a.H + k0, a.H, t.rows);
        const int64_t wo = (int64_t)k0 * a.I + i0;
        wl.init(a.w0 + wo, a.I, a.H - k0, a.I - i0, a.w1 + wo);
        nk = min(a.len, a.H / C::BK - t.s * a.len);
        return true;
    }
    __device__ void issue(int kt, uint32_t tile) {
        xl.issue(kt * C::BK, tile);
        wl.issue(kt * C::BK, tile + C::X_BYTES);
    }
    // gate block fn pairs with up block fn + FN/2 inside the same wave
    __device__ int wrow(int wn, int fn) const {
        return fn < C::FN / 2 ? wn * (C::WN / 2) + fn * 32 : C::BN / 2 + wn * (C::WN / 2) + (fn - C::FN / 2) * 32;
    }
    __device__ void epilogue(f32x16_t (&acc)[C::FM][C::FN], int wm, int wn) {
        using FS = FragStage<C, C::LDS_BYTES>;
        const int I = a.I, ib = i0 + wn * (C::WN / 2);
        const bool live = ib < I;   // I % 64 == 0: the wave's i are all valid or all past I
        if (a.splits > 1) {
            store_partials<C>(acc, a.part + ((int64_t)t.s * a.T + t.m0) * 2 * I, 2 * I, t.rows, wm, live, [&](int fn) {
                return fn < C::FN / 2 ? ib + fn * 32 : I + ib + (fn - C::FN / 2) * 32;
            });
            return;
        }
        if (!live) return;
        const int lane = epi_lane();
        const uint32_t area = FS::area(wave_id(), 1);
        // a, K-tiled for the down product's loads: [I/32][T][32], so that a
        // K-step of a tile's rows is one contiguous run
        const brsrc_t adst = rows_rsrc(a.a, (uint32_t)((int64_t)a.T * I * 2));
        const uint32_t a0 = (uint32_t)(ib / 32) * (uint32_t)a.T * 64u + (uint32_t)t.m0 * 64u;
#pragma unroll
        for (int fm = 0; fm < C::FM; ++fm) {
#pragma unroll
            for (int fn = 0; fn < C::FN / 2; ++fn)
#pragma unroll
                for (int g4 = 0; g4 < 4; ++g4) {
                    float v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float hg = acc[fm][fn][g4 * 4 + j], hu = acc[fm][fn + C::FN / 2][g4 * 4 + j];
                        v[j] = hg * sigmoidf_(hg) * hu;
                    }
                    FS::put(area + FS::frag_off(fn, g4, lane),
                            pack4(v[0], v[1], v[2], v[3]));
                }
            // the first half of each staged row: 32 values of i; the other lanes store nothing
#pragma unroll
            for (int p = 0; p < FS::PASSES; ++p) {
                const int m = wm * C::WM + fm * 32 + FS::pass_row(p, lane), cc = FS::pass_col(lane);
                const bool ok = m < t.rows && cc < C::WN / 2;
                bstore8_nt(adst, ok ? a0 + (uint32_t)m * 64u + 2u * (uint32_t)cc : kOutOfRange, 0,
                           FS::get(area + FS::pass_off(p, lane)));
            }
        }
        if (!a.h) return;
        // gate columns go to h[.., i], up columns to h[.., I + i]
        const uint32_t h_row = 4u * (uint32_t)I;
        const uint32_t h_col = 2u * (uint32_t)(ib + (FS::pass_col(lane) >= C::WN / 2 ? I - C::WN / 2 : 0));
        staged_rows<C, C::LDS_BYTES>([&](int fm, int fn, int g4, int j) { return acc[fm][fn][g4 * 4 + j]; },
                                     rows_rsrc(a.h + (int64_t)t.m0 * 2 * I, (uint32_t)t.rows * h_row),
                                     [&](int fm, int r) -> uint32_t {
                                         return (uint32_t)(wm * C::WM + fm * 32 + r) * h_row + h_col;
                                     });
    }
};

// out = addend + a W_down
template <class Cfg>
struct FfnDown {
    using C = Cfg;
    using Args = FfnArgs;
    static constexpr bool X_TRANS = false, W_TRANS = true;
    RowLoader<C, C::BM> xl;
    TransLoader<C, C::BN> wl;
    static constexpr int LOADS_PER_STAGE = RowLoader<C, C::BM>::IPW + TransLoader<C, C::BN>::IPW;
    FfnTile t;
    int nk;
    Args a;
    __device__ int mvalid() const { return t.rows; }

    __device__ bool setup(const Args &args, int b) {
        a = args;
        if (!ffn_tile(a.T, C::BM, a.n_tiles, a.splits, b, t)) return false;
        const int s0 = t.s * a.len, n0 = t.nt * C::BN;   // s0: first K-step, one 32-column block of a each
        const int64_t off = ((int64_t)s0 * a.T + t.m0) * 32;
        xl.init_tiled(a.x + off, (uint32_t)a.T * 64u, (uint32_t)((int64_t)a.T * a.I * 2 - off * 2));
        wl.init(a.w0 + (int64_t)s0 * C::BK * a.H + n0, a.H, a.I - s0 * C::BK, a.H - n0);
        nk = min(a.len, a.I / C::BK - s0);
        return true;
    }
    __device__ void issue(int kt, uint32_t tile) {
        xl.issue(kt * C::BK, tile);
        wl.issue(kt * C::BK, tile + C::X_BYTES);
    }
    __device__ int wrow(int wn, int fn) const { return wn * C::WN + fn * 32; }
    __device__ void epilogue(f32x16_t (&acc)[C::FM][C::FN], int wm, int wn) {
        dense_epilogue<C, C::LDS_BYTES>(acc, t, a.T, a.H, a.splits, wm, wn, a.addend, a.out, a.part);
    }
};

// G = dy W_down^T with the SwiGLU backward: dh, and a for dW_down
template <class Cfg>
struct FfnDA {
    using C = Cfg;
    using Args = FfnArgs;
    static constexpr bool X_TRANS = false, W_TRANS = false;
    RowLoader<C, C::BM> xl;
    RowLoader<C, C::BN> wl;
    static constexpr int LOADS_PER_STAGE = RowLoader<C, C::BM>::IPW + RowLoader<C, C::BN>::IPW;
    FfnTile t;
    int nk;
    Args a;
    __device__ int mvalid() const { return t.rows; }

    __device__ bool setup(const Args &args, int b) {
        a = args;
        if (!ffn_tile(a.T, C::BM, a.n_tiles, a.splits, b, t)) return false;
        const int k0 = t.s * a.len * C::BK, i0 = t.nt * C::BN;
        xl.init(a.x + (int64_t)t.m0 * a.H + k0, a.H, t.rows);
        wl.init(a.w0 + (int64_t)i0 * a.H + k0, a.H, min(C::BN, a.I - i0));
        nk = min(a.len, a.H / C::BK - t.s * a.len);
        return true;
    }
    __device__ void issue(int kt, uint32_t tile) {
        xl.issue(kt * C::BK, tile);
        wl.issue(kt * C::BK, tile + C::X_BYTES);
    }
    __device__ int wrow(int wn, int fn) const { return wn * C::WN + fn * 32; }
    // h rows come in and dh and a rows leave as whole row runs, staged one
    // 32-row fragment at a time
    __device__ void epilogue(f32x16_t (&acc)[C::FM][C::FN], int wm, int wn) {
        using FS = FragStage<C, C::LDS_BYTES>;
        const int I = a.I, ib0 = t.nt * C::BN + wn * C::WN;
        const bool live = ib0 < I;
        if (a.splits > 1) {
            store_partials<C>(acc, a.part + ((int64_t)t.s * a.T + t.m0) * I, I, t.rows, wm, live,
                              [&](int fn) { return ib0 + fn * 32; });
            return;
        }
        const int lane = epi_lane();
        const int ib = live ? ib0 : 0;
        const uint32_t rows = live ? (uint32_t)t.rows : 0u;
        const uint32_t sg = FS::area(wave_id(), 3), su = sg + FS::BYTES, sa = su + FS::BYTES;
        const uint32_t row_bytes = 4u * (uint32_t)I, up = 2u * (uint32_t)I;
        const brsrc_t hres = rows_rsrc(a.h_in + (int64_t)t.m0 * 2 * I, rows * row_bytes);
        const brsrc_t dres = rows_rsrc(a.dh + (int64_t)t.m0 * 2 * I, rows * row_bytes);
        const brsrc_t ares = rows_rsrc(a.a + (int64_t)t.m0 * I, rows * up);
        auto row = [&](int fm, int p) { return (uint32_t)(wm * C::WM + fm * 32 + FS::pass_row(p, lane)); };
        const uint32_t col = 2u * (uint32_t)(ib + FS::pass_col(lane));
        uint2 hg[FS::PASSES], hu[FS::PASSES];
        auto load_h = [&](int fm) {
#pragma unroll
            for (int p = 0; p < FS::PASSES; ++p) {
                hg[p] = bload8(hres, row(fm, p) * row_bytes + col, 0);
                hu[p] = bload8(hres, row(fm, p) * row_bytes + col, up);
            }
        };
        load_h(0);
#pragma unroll
        for (int fm = 0; fm < C::FM; ++fm) {
#pragma unroll
            for (int p = 0; p < FS::PASSES; ++p) {
                FS::put(sg + FS::pass_off(p, lane), hg[p]);
                FS::put(su + FS::pass_off(p, lane), hu[p]);
            }
            __builtin_amdgcn_sched_barrier(0);   // phases stay in order: keeps live ranges short
#pragma unroll
            for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
                for (int g4 = 0; g4 < 4; ++g4) {
                    const uint32_t o = FS::frag_off(fn, g4, lane);
                    const uint2 hg2 = FS::get(sg + o), hu2 = FS::get(su + o);
                    GluGrad r[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        r[j] = glu_backward(acc[fm][fn][g4 * 4 + j], bf16_at(hg2, j), bf16_at(hu2, j));
                    FS::put(sg + o, pack4(r[0].dg, r[1].dg, r[2].dg, r[3].dg));
                    FS::put(su + o, pack4(r[0].du, r[1].du, r[2].du, r[3].du));
                    FS::put(sa + o, pack4(r[0].a, r[1].a, r[2].a, r[3].a));
                }
            __builtin_amdgcn_sched_barrier(0);
            if (fm + 1 < C::FM) load_h(fm + 1);   // in flight while this fragment's rows are stored
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int p = 0; p < FS::PASSES; ++p) {
                const uint32_t o = FS::pass_off(p, lane), v = row(fm, p) * row_bytes + col;
                bstore8_nt(dres, v, 0, FS::get(sg + o));
                bstore8_nt(dres, v, up, FS::get(su + o));
                bstore8_nt(ares, row(fm, p) * up + col, 0, FS::get(sa + o));
            }
        }
    }
};

// dx = addend + dh_g W_gate^T + dh_u W_up^T
template <class Cfg>
struct FfnDX {
    using C = Cfg;
    using Args = FfnArgs;
    static constexpr bool X_TRANS = false, W_TRANS = false;
    RowLoader<C, C::BM> xl;
    RowLoader<C, C::BN> wl;
    static constexpr int LOADS_PER_STAGE = RowLoader<C, C::BM>::IPW + RowLoader<C, C::BN>::IPW;
    FfnTile t;
    int nk;
    Args a;
    __device__ int mvalid() const { return t.rows; }

    __device__ bool setup(const Args &args, int b) {
        a = args;
        if (!ffn_tile(a.T, C::BM, a.n_tiles, a.splits, b, t)) return false;
        const int I = a.I, k0 = t.s * a.len * C::BK, n0 = t.nt * C::BN, nw = min(C::BN, a.H - n0);
        xl.init(a.x + (int64_t)t.m0 * 2 * I + k0, 2 * I, t.rows);
        const int64_t wo = (int64_t)n0 * I;
        if (k0 < I)   // the run starts among the gate columns and may go on into the up columns
            wl.init(a.w0 + wo + k0, I, nw, a.w1 + wo, I - k0);
        else
            wl.init(a.w1 + wo + (k0 - I), I, nw);
        nk = min(a.len, 2 * I / C::BK - t.s * a.len);
        return true;
    }
    __device__ void issue(int kt, uint32_t tile) {
        xl.issue(kt * C::BK, tile);
        wl.issue(kt * C::BK, tile + C::X_BYTES);
    }
    __device__ int wrow(int wn, int fn) const { return wn * C::WN + fn * 32; }
    __device__ void epilogue(f32x16_t (&acc)[C::FM][C::FN], int wm, int wn) {
        dense_epilogue<C, C::LDS_BYTES>(acc, t, a.T, a.H, a.splits, wm, wn, a.addend, a.out, a.part);
    }
};

template <class P>
__global__ __launch_bounds__(P::C::NT, P::C::OCC) void ffn_gemm(typename P::Args args) {
    extern __shared__ __attribute__((aligned(1024))) char lds_raw[];
    P p;
    if (!p.setup(args, (int)blockIdx.x)) return;
    gemm_tile(p, (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds_raw);
}

// dW_gate | dW_up, dW_down and dx in one launch, the weight gradients (the
// longer K loops) first; g0, g1: workgroups of the first two.
template <class PX, class PW>
__global__ __launch_bounds__(PX::C::NT, PX::C::OCC) void ffn_grads(typename PW::Args gu, typename PW::Args wd,
                                                          typename PX::Args ax, int g0, int g1) {
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
        gemm_tile(p, lds);
    }
}

template <class P>
hipError_t launch_product(const char *name, unsigned grid, const FfnArgs &a, hipStream_t st) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds(ffn_gemm<P>, P::C::LDS_BYTES, done);
    if (e != hipSuccess) return e;
    KernelTimer tm(name, st);
    ffn_gemm<P><<<grid, P::C::NT, P::C::LDS_BYTES, st>>>(a);
    return hipGetLastError();
}

template <template <class> class P>
hipError_t product(const char *name, const FfnSplit &s, FfnArgs a, int n_tiles, hipStream_t st) {
    a.n_tiles = n_tiles;
    a.splits = s.splits;
    a.len = s.len;
    const unsigned grid = ffn_grid(a.T, s.bm, n_tiles, s.splits);
    return s.bm == CfgS::BM ? launch_product<P<CfgS>>(name, grid, a, st) : launch_product<P<CfgA>>(name, grid, a, st);
}

template <class CX, class CW>
hipError_t launch_grads(const FfnWgradArgs &gu, const FfnWgradArgs &wd, const FfnArgs &ax, hipStream_t st) {
    static std::atomic<uint64_t> done{0};
    auto *k = ffn_grads<FfnDX<CX>, FfnWgrad<CW>>;
    constexpr size_t lds = CX::LDS_BYTES > CW::LDS_BYTES ? CX::LDS_BYTES : CW::LDS_BYTES;
    const hipError_t e = allow_lds(k, lds, done);
    if (e != hipSuccess) return e;
    const unsigned g0 = wgrad_grid(gu.M, gu.N, CW::BM), g1 = wgrad_grid(wd.M, wd.N, CW::BM);
    const unsigned gx = ffn_grid(ax.T, CX::BM, ax.n_tiles, ax.splits);
    KernelTimer tm("ffn_grads", st);
    k<<<g0 + g1 + gx, CX::NT, lds, st>>>(gu, wd, ax, (int)g0, (int)g1);
    return hipGetLastError();
}

hipError_t forward_bf16(const FfnPlan &p, char *ws, const uint16_t *x, const mok_weights &w, const uint16_t *addend,
                        uint16_t *out, uint16_t *h, hipStream_t st) {
    FfnArgs a{};
    a.T = (int)p.T;
    a.H = p.H;
    a.I = p.I;
    a.x = x;
    a.w0 = static_cast<const uint16_t *>(w.w_gate);
    a.w1 = static_cast<const uint16_t *>(w.w_up);
    a.h = h;
    a.a = reinterpret_cast<uint16_t *>(ws + p.a);
    a.part = reinterpret_cast<float *>(ws + p.part);
    hipError_t e = product<FfnGateUp>("ffn_gate_up", p.gate_up, a, (int)ceil_div(p.I, kTileN / 2), st);
    if (e != hipSuccess) return e;
    if (p.gate_up.splits > 1) {
        KernelTimer tm("ffn_join_act", st);
        ffn_join_act<false><<<join_grid(p.T, p.I), 256, 0, st>>>(a.part, p.gate_up.splits, a.T, a.I, h, a.a, nullptr,
                                                                 nullptr);
    }
    a.x = a.a;
    a.w0 = static_cast<const uint16_t *>(w.w_down);
    a.addend = addend;
    a.out = out;
    e = product<FfnDown>("ffn_down", p.down, a, (int)ceil_div(p.H, kTileN), st);
    if (e == hipSuccess && p.down.splits > 1) {
        KernelTimer tm("ffn_join_out", st);
        ffn_join_out<<<join_grid(p.T, p.H), 256, 0, st>>>(a.part, p.down.splits, a.T, a.H, addend, out);
        e = hipGetLastError();
    }
    return e;
}

hipError_t backward_bf16(const FfnPlan &p, char *ws, const uint16_t *x, const mok_weights &w, const uint16_t *h,
                         const uint16_t *dy, const uint16_t *addend, uint16_t *dx, uint16_t *dw_gate, uint16_t *dw_up,
                         uint16_t *dw_down, hipStream_t st) {
    FfnArgs a{};
    a.T = (int)p.T;
    a.H = p.H;
    a.I = p.I;
    a.a = reinterpret_cast<uint16_t *>(ws + p.a);
    a.dh = reinterpret_cast<uint16_t *>(ws + p.dh);
    a.part = reinterpret_cast<float *>(ws + p.part);
    hipError_t e = hipSuccess;
    if (p.T > 0) {
        a.x = dy;
        a.w0 = static_cast<const uint16_t *>(w.w_down);
        a.h_in = h;
        e = product<FfnDA>("ffn_da", p.da, a, (int)ceil_div(p.I, kTileN), st);
        if (e != hipSuccess) return e;
        if (p.da.splits > 1) {
            KernelTimer tm("ffn_join_da", st);
            ffn_join_da<false><<<join_grid(p.T, p.I), 256, 0, st>>>(a.part, p.da.splits, a.T, a.I, h, a.dh, a.a,
                                                                    nullptr, nullptr);
        }
    }
    a.x = a.dh;
    a.w0 = static_cast<const uint16_t *>(w.w_gate);
    a.w1 = static_cast<const uint16_t *>(w.w_up);
    a.addend = addend;
    a.out = dx;
    a.n_tiles = (int)ceil_div(p.H, kTileN);
    a.splits = p.dx.splits;
    a.len = p.dx.len;
    const FfnWgradArgs gu{a.T, p.H, 2 * p.I, p.I, p.I, x, a.dh, dw_gate, dw_up};
    const FfnWgradArgs wd{a.T, p.I, p.H, p.H, p.H, a.a, dy, dw_down, nullptr};
    if (p.grads_two)
        e = launch_grads<CfgW, CfgW>(gu, wd, a, st);
    else if (p.dx.bm == CfgS::BM)
        e = p.wgrad_bm == CfgS::BM ? launch_grads<CfgS, CfgS>(gu, wd, a, st) : launch_grads<CfgS, CfgA>(gu, wd, a, st);
    else
        e = p.wgrad_bm == CfgS::BM ? launch_grads<CfgA, CfgS>(gu, wd, a, st) : launch_grads<CfgA, CfgA>(gu, wd, a, st);
    if (e == hipSuccess && p.T > 0 && p.dx.splits > 1) {
        KernelTimer tm("ffn_join_out", st);
        ffn_join_out<<<join_grid(p.T, p.H), 256, 0, st>>>(a.part, p.dx.splits, a.T, a.H, addend, dx);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace

hipError_t ffn_mx_forward(const FfnPlan &p, char *ws, const uint8_t *x_elems, const uint8_t *x_scales,
                          const mok_weights &w, const uint16_t *addend, uint16_t *out, uint16_t *h, hipStream_t st);
hipError_t ffn_mx_backward(const FfnPlan &p, char *ws, const uint16_t *x, const mok_weights &w, const uint16_t *h,
                           const uint16_t *dy, const uint16_t *addend, uint16_t *dx, uint16_t *dw_gate, uint16_t *dw_up,
                           uint16_t *dw_down, hipStream_t st);

mok_status launch_ffn_forward(const FfnPlan &p, void *workspace, const uint16_t *x, const uint8_t *x_elems,
                              const uint8_t *x_scales, const mok_weights &w, const uint16_t *addend, uint16_t *out,
                              uint16_t *h, hipStream_t st) {
    char *ws = static_cast<char *>(workspace);
    hipError_t e;
    if (p.few_runs)
        e = p.mx ? ffn_few_mx_forward(p, ws, x_elems, x_scales, w, addend, out, h, st)
                 : ffn_few_forward(p, ws, x, w, addend, out, h, st);
    else
        e = p.mx ? ffn_mx_forward(p, ws, x_elems, x_scales, w, addend, out, h, st)
                 : forward_bf16(p, ws, x, w, addend, out, h, st);
    return check_hip(e, "mok_ffn_forward");
}

mok_status launch_ffn_backward(const FfnPlan &p, void *workspace, const uint16_t *x, const mok_weights &w,
                               const uint16_t *h, const uint16_t *dy, const uint16_t *addend, uint16_t *dx,
                               uint16_t *dw_gate, uint16_t *dw_up, uint16_t *dw_down, hipStream_t st) {
    char *ws = static_cast<char *>(workspace);
    const hipError_t e = p.mx ? ffn_mx_backward(p, ws, x, w, h, dy, addend, dx, dw_gate, dw_up, dw_down, st)
                              : backward_bf16(p, ws, x, w, h, dy, addend, dx, dw_gate, dw_up, dw_down, st);
    return check_hip(e, "mok_ffn_backward");
}

}  // namespace mok
