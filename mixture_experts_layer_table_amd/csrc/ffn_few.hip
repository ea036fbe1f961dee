// Gated feed-forward block for a few rows (single-token decoding): forward
// only, at most kFewRows rows.
//
// Bound by reading the weights once (7,168 x 2,048 in BF16: 88 MB, 17 us at the
// 5.2 TB/s of a large copy): no matrix core, no LDS staging of weights, each
// lane multiplies the 16 bytes it loads with fp32 fused multiply-adds. The tile
// kernels need four launches here (both products split over their contraction
// axis, both joined); this form needs two:
//   1. gate/up, the contraction axis cut into few enough runs that the second
//      kernel can add them itself (BF16), or not cut at all (MXFP8, whose
//      weights are contiguous along it);
//   2. down: every workgroup makes a = silu(h_g) h_u for itself, asked for ahead
//      of its weights, then finishes whole outputs.
// a stays in fp32 in BF16 mode (one rounding fewer than the tile kernels).
// Sums run in a fixed order: lane, wave, run.
//
// Measured, one row of 7,168 x 2,048: BF16 23 to 25 us over several cards (gate/up
// 13, down 10), MXFP8 16 (9 and 6), two rows in MXFP8 21. Each kernel's
// launch, first loads and lane sums are 4 to 5 us.
//
// Which calls come here is plan_few's rule (ffn_plan.cpp). The cost that grows
// with the rows is each lane's sums, not the weights: at 7,168 x 2,048 two BF16
// rows take 32 us here and 29 on the tiles, four 38 and 29.
#include "ffn_few.h"
#include "ffn_parts.h"
#include "kernels.h"
#include "lanes.h"

namespace mok {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kBatch = 16;   // weight loads of one array in flight per lane

__device__ __forceinline__ void unpack_bf16x8(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

// Weights are read once: keep them from displacing what is read again.
__device__ __forceinline__ uint4 load_once(const void *p) {
    typedef uint32_t v4u __attribute__((ext_vector_type(4)));
    const v4u v = __builtin_nontemporal_load(static_cast<const v4u *>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}

// 16 bytes at byte voff + soff (soff uniform) of a range; past it: zeros, with
// no branch (gfx950 checks the sum of both offsets, also where soff alone lies past
// the range: held on a buffer whose memory goes on behind the range). Cached: two
// workgroups share each line of W_down (non-temporal, the down kernel took 12.3 us
// instead of 10.7 at 7,168 x 2,048).
__device__ __forceinline__ uint4 load16(brsrc_t r, uint32_t voff, uint32_t soff) {
    typedef uint32_t v4u __attribute__((ext_vector_type(4)));
    const v4u v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, 0);
    return make_uint4(v.x, v.y, v.z, v.w);
}

// ----------------------------------------------------------------------------- BF16

struct FewArgs {
    int H, I, runs, run_rows;   // run_rows: rows of W_gate / W_up in one run, a multiple of 64
    const uint16_t *x, *wg, *wu, *wd, *addend;
    uint16_t *out, *h;
    float *part;   // [runs][T][2I]
};

// One strip of 64 gate and the same 64 up columns over one run: 8 lanes cover
// the strip's 128-byte row piece, a wave 8 rows a load, the workgroup 64.
template <int T>
__global__ __launch_bounds__(kThreads, 2) void few_gate_up(FewArgs a, int rows) {
    extern __shared__ __attribute__((aligned(16))) float few_lds[];
    const int strips = a.I / 64, strip = (int)blockIdx.x % strips, run = (int)blockIdx.x / strips;
    const int k0 = run * a.run_rows, kn = min(a.run_rows, a.H - k0), n = kn / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, cg = lane & 7, r0 = wave * 8 + (lane >> 3);
    float *xs = few_lds, *red = few_lds + T * a.run_rows;   // x [T][run_rows]; [waves][T][128]
    const uint32_t bytes = (uint32_t)((int64_t)kn * a.I * 2), step = (uint32_t)(64 * a.I * 2);
    const brsrc_t g = rows_rsrc(a.wg + (int64_t)k0 * a.I, bytes), u = rows_rsrc(a.wu + (int64_t)k0 * a.I, bytes);
    const uint32_t v0 = (uint32_t)(r0 * a.I + strip * 64 + cg * 8) * 2u;
    float sg[T][8], su[T][8];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) sg[t][j] = su[t][j] = 0.0f;
    // x is asked for ahead of the weights: loads return in order
    auto x4 = [&](int e) {   // 4 values at flat position e of the run's x [T][kn]
        const int t = e / kn, k = e - t * kn;
        return t < rows ? *reinterpret_cast<const uint2 *>(a.x + (int64_t)t * a.H + k0 + k) : make_uint2(0, 0);
    };
    auto put_x4 = [&](int e, uint2 v) {
        const int t = e / kn, k = e - t * kn;
        *reinterpret_cast<f32x4_t *>(xs + t * a.run_rows + k) =
            f32x4_t{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
    };
    const int e0 = (int)threadIdx.x * 4;
    uint2 x0 = make_uint2(0, 0);
    if (e0 < T * kn) x0 = x4(e0);
    for (int b = 0; b < n; b += kBatch) {
        uint4 gv[kBatch], uv[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {   // rows past the run: zeros
            gv[i] = load16(g, v0, (uint32_t)(b + i) * step);
            uv[i] = load16(u, v0, (uint32_t)(b + i) * step);
        }
        if (b == 0) {
            if (e0 < T * kn) put_x4(e0, x0);
            for (int e = e0 + kThreads * 4; e < T * kn; e += kThreads * 4) put_x4(e, x4(e));
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (b + i < n) {
                float gf[8], uf[8];
                unpack_bf16x8(gv[i], gf);
                unpack_bf16x8(uv[i], uf);
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    const float xv = xs[t * a.run_rows + (b + i) * 64 + r0];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        sg[t][j] = __builtin_fmaf(xv, gf[j], sg[t][j]);
                        su[t][j] = __builtin_fmaf(xv, uf[j], su[t][j]);
                    }
                }
            }
    }
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float vg = sum_lanes<8>(sg[t][j]), vu = sum_lanes<8>(su[t][j]);
            if (lane < 8) {
                red[(wave * T + t) * 128 + cg * 8 + j] = vg;
                red[(wave * T + t) * 128 + 64 + cg * 8 + j] = vu;
            }
        }
    __syncthreads();
    for (int e = threadIdx.x; e < T * 128; e += kThreads) {
        const int t = e / 128, c = e % 128;
        if (t >= rows) break;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += red[(w * T + t) * 128 + c];
        a.part[((int64_t)run * rows + t) * 2 * a.I + (c < 64 ? 0 : a.I - 64) + strip * 64 + c] = s;
    }
}

// a at flat position e (row e / I, 4 values of i) in two steps: the loads of the
// first kJoinBatch runs' partials, then their sums, the rest of the runs and the
// activation. save: also write h.
__device__ __forceinline__ void load_runs(const FewArgs &a, int rows, int e, f32x4_t (&hg)[kJoinBatch],
                                          f32x4_t (&hu)[kJoinBatch]) {
    const int t = e / a.I, i = e - t * a.I;
    if (t >= rows) return;
    const float *p = a.part + (int64_t)t * 2 * a.I + i;
    const int64_t stride = (int64_t)rows * 2 * a.I;
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j) {
        hg[j] = *reinterpret_cast<const f32x4_t *>(p + min(j, a.runs - 1) * stride);
        hu[j] = *reinterpret_cast<const f32x4_t *>(p + a.I + min(j, a.runs - 1) * stride);
    }
}
__device__ __forceinline__ f32x4_t act_of(const FewArgs &a, int rows, int e, const f32x4_t (&hg)[kJoinBatch],
                                          const f32x4_t (&hu)[kJoinBatch], bool save) {
    const int t = e / a.I, i = e - t * a.I;
    if (t >= rows) return f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    f32x4_t g = hg[0], u = hu[0], v;
#pragma unroll
    for (int j = 1; j < kJoinBatch; ++j)
        if (j < a.runs) {
            g += hg[j];
            u += hu[j];
        }
    const float *p = a.part + (int64_t)t * 2 * a.I + i;
    for (int j = kJoinBatch; j < a.runs; ++j) {
        g += *reinterpret_cast<const f32x4_t *>(p + (int64_t)j * rows * 2 * a.I);
        u += *reinterpret_cast<const f32x4_t *>(p + a.I + (int64_t)j * rows * 2 * a.I);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = g[j] * sigmoidf_(g[j]) * u[j];
    if (a.h && save) {
        *reinterpret_cast<uint2 *>(a.h + (int64_t)t * 2 * a.I + i) = pack4(g[0], g[1], g[2], g[3]);
        *reinterpret_cast<uint2 *>(a.h + (int64_t)t * 2 * a.I + a.I + i) =
            pack4(u[0], u[1], u[2], u[3]);
    }
    return v;
}

// One strip of 32 output columns over the whole contraction axis: 4 lanes cover
// the strip's 64-byte row piece, a wave 16 rows a load. Two neighbouring strips
// share each 128-byte line and run on one XCD.
template <int T>
__global__ __launch_bounds__(kThreads, 2) void few_down(FewArgs a, int rows) {
    extern __shared__ __attribute__((aligned(16))) float few_lds[];
    const int idx = (int)blockIdx.x / kXcds, strip = (idx / 2 * kXcds + (int)blockIdx.x % kXcds) * 2 + (idx & 1);
    if (strip >= a.H / 32) return;
    const int I = a.I, n = (I + 127) / 128;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, cg = lane & 3, r0 = wave * 16 + (lane >> 2);
    float *as = few_lds, *red = few_lds + T * I;   // a [T][I]; [waves][T][32]
    const brsrc_t w = rows_rsrc(a.wd, (uint32_t)((int64_t)I * a.H * 2));
    const uint32_t v0 = (uint32_t)(r0 * a.H + strip * 32 + cg * 8) * 2u, step = (uint32_t)(128 * a.H * 2);
    float acc[T][8];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t][j] = 0.0f;
    // The first 4 values of i of each thread are asked for ahead of the weights
    // (loads return in order), so that a is ready when the weights arrive.
    const int e0 = (int)threadIdx.x * 4;
    f32x4_t hg[kJoinBatch], hu[kJoinBatch];
    if (e0 < T * I) load_runs(a, rows, e0, hg, hu);
    for (int b = 0; b < n; b += kBatch) {
        uint4 wv[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) wv[i] = load16(w, v0, (uint32_t)(b + i) * step);   // rows past I: zeros
        if (b == 0) {
            for (int e = e0; e < T * I; e += kThreads * 4) {
                if (e != e0) load_runs(a, rows, e, hg, hu);
                *reinterpret_cast<f32x4_t *>(as + e) = act_of(a, rows, e, hg, hu, strip == 0);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = (b + i) * 128 + r0;
            if (b + i < n) {
                float f[8];
                unpack_bf16x8(wv[i], f);
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    const float av = k < I ? as[t * I + k] : 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[t][j] = __builtin_fmaf(av, f[j], acc[t][j]);
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = sum_lanes<4>(acc[t][j]);
            if (lane < 4) red[(wave * T + t) * 32 + cg * 8 + j] = v;
        }
    __syncthreads();
    const int e = threadIdx.x, t = e / 32;
    if (e < T * 32 && t < rows) {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) s += red[v * T * 32 + e];
        const int64_t o = (int64_t)t * a.H + strip * 32 + e % 32;
        if (a.addend) s += bf16_to_f32(a.addend[o]);
        a.out[o] = (uint16_t)f32_to_bf16(s);
    }
}

// ----------------------------------------------------------------------------- MXFP8

// The values of 4 E4M3 codes.
__device__ __forceinline__ f32x4_t unpack_fp8x4(uint32_t w) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return f32x4_t{lo.x, lo.y, hi.x, hi.y};
}
__device__ __forceinline__ void unpack_fp8x16(const uint4 &v, float (&f)[16]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x4_t u = unpack_fp8x4(w[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[4 * i + j] = u[j];
    }
}

struct Few8Args {
    int H, I, lanes;   // lanes that share a weight row, 16 values each: a power of two, at most 64
    const uint8_t *x, *xs, *wg, *wgs, *wu, *wus, *wd, *wds;
    const uint16_t *addend;
    uint16_t *out, *h;
    float *act;   // a [T][I] before its quantization
};

constexpr int kBatch8 = 7;   // 16-byte pieces of a row in flight per lane

// One (gate, up) pair of weight rows per group of lanes: h, and a in fp32.
template <int T>
__global__ __launch_bounds__(kThreads, 2) void few_gate_up8(Few8Args a, int rows) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, per = 64 / a.lanes, l = lane % a.lanes;
    const int i = ((int)blockIdx.x * kWaves + wave) * per + lane / a.lanes;
    const bool ok = i < a.I;
    const int row = ok ? i : 0, H = a.H, n = (H + 16 * a.lanes - 1) / (16 * a.lanes);
    const uint8_t *g = a.wg + (int64_t)row * H, *u = a.wu + (int64_t)row * H;
    const uint8_t *gs = a.wgs + (int64_t)row * (H / 32), *us = a.wus + (int64_t)row * (H / 32);
    float sg[T], su[T];
#pragma unroll
    for (int t = 0; t < T; ++t) sg[t] = su[t] = 0.0f;
    for (int b = 0; b < n; b += kBatch8) {
        uint4 gv[kBatch8], uv[kBatch8], xv[T][kBatch8];
        uint32_t ge[kBatch8], ue[kBatch8], xe[T][kBatch8];
#pragma unroll
        for (int c = 0; c < kBatch8; ++c) {
            const int k = ((b + c) * a.lanes + l) * 16;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                xv[t][c] = make_uint4(0, 0, 0, 0);
                xe[t][c] = 127;
                if (k < H && t < rows) {
                    xv[t][c] = *reinterpret_cast<const uint4 *>(a.x + (int64_t)t * H + k);
                    xe[t][c] = a.xs[(int64_t)t * (H / 32) + k / 32];
                }
            }
            gv[c] = uv[c] = make_uint4(0, 0, 0, 0);
            ge[c] = ue[c] = 127;
            if (k < H) {
                gv[c] = load_once(g + k);
                uv[c] = load_once(u + k);
                ge[c] = gs[k / 32];
                ue[c] = us[k / 32];
            }
        }
#pragma unroll
        for (int c = 0; c < kBatch8; ++c) {
            if ((b + c) * a.lanes * 16 >= H) break;   // the same for every lane; a lane past H holds zeros
            float gf[16], uf[16];
            unpack_fp8x16(gv[c], gf);
            unpack_fp8x16(uv[c], uf);
#pragma unroll
            for (int t = 0; t < T; ++t) {
                float xf[16];
                unpack_fp8x16(xv[t][c], xf);
                float dg = 0.0f, du = 0.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    dg = __builtin_fmaf(gf[j], xf[j], dg);
                    du = __builtin_fmaf(uf[j], xf[j], du);
                }
                // half of one 32-block; the two scales as one exponent, so that neither
                // alone can over- or underflow a sum whose value is in range
                sg[t] += __builtin_ldexpf(dg, (int)(ge[c] + xe[t][c]) - 254);
                su[t] += __builtin_ldexpf(du, (int)(ue[c] + xe[t][c]) - 254);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const float hg = sum_group(sg[t], a.lanes), hu = sum_group(su[t], a.lanes);
        if (l == 0 && ok && t < rows) {
            a.act[(int64_t)t * a.I + i] = hg * sigmoidf_(hg) * hu;
            if (a.h) {
                a.h[(int64_t)t * 2 * a.I + i] = (uint16_t)f32_to_bf16(hg);
                a.h[(int64_t)t * 2 * a.I + a.I + i] = (uint16_t)f32_to_bf16(hu);
            }
        }
    }
}

constexpr int kRowsPerGroup = 4;   // output columns (weight rows) per group of lanes

template <int T>
__global__ __launch_bounds__(kThreads, 2) void few_down8(Few8Args a, int rows) {
    extern __shared__ __attribute__((aligned(16))) float few_lds[];   // what a's codes hold, without their scales: [T][I]
    const int I = a.I, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, per = 64 / a.lanes, l = lane % a.lanes;
    const int n0 = (((int)blockIdx.x * kWaves + wave) * per + lane / a.lanes) * kRowsPerGroup;
    const int n = (I + 16 * a.lanes - 1) / (16 * a.lanes);
    uint32_t *as = reinterpret_cast<uint32_t *>(few_lds + T * I);   // a's scale bytes, [T][I / 32]
    float acc[T][kRowsPerGroup];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < kRowsPerGroup; ++r) acc[t][r] = 0.0f;
    auto act4 = [&](int e) {
        const int t = e / I;
        return t < rows ? *reinterpret_cast<const f32x4_t *>(a.act + e) : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    };
    const int e0 = (int)threadIdx.x * 4;
    f32x4_t a0 = {0.0f, 0.0f, 0.0f, 0.0f};   // asked for ahead of the weights
    if (e0 < T * I) a0 = act4(e0);
    for (int c = 0; c < n; ++c) {
        const int k = (c * a.lanes + l) * 16;
        uint4 wv[kRowsPerGroup];
        uint32_t we[kRowsPerGroup];
#pragma unroll
        for (int r = 0; r < kRowsPerGroup; ++r) {
            wv[r] = make_uint4(0, 0, 0, 0);
            we[r] = 127;
            if (k < I && n0 + r < a.H) {
                wv[r] = load_once(a.wd + (int64_t)(n0 + r) * I + k);
                we[r] = a.wds[(int64_t)(n0 + r) * (I / 32) + k / 32];
            }
        }
        if (c == 0) {
            for (int e = e0; e < T * I; e += kThreads * 4) {   // whole 32-blocks per 8 lanes
                const f32x4_t p = e == e0 ? a0 : act4(e);
                const float v[4] = {p[0], p[1], p[2], p[3]};
                uint32_t sc;
                const uint32_t code = quantize_lane4(v, sc);
                *reinterpret_cast<f32x4_t *>(few_lds + e) = unpack_fp8x4(code);
                if (e % 32 == 0) as[e / 32] = sc;
            }
            __syncthreads();
        }
        if (k < I) {
#pragma unroll
            for (int r = 0; r < kRowsPerGroup; ++r) {
                float f[16];
                unpack_fp8x16(wv[r], f);
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    float d = 0.0f;
#pragma unroll
                    for (int j4 = 0; j4 < 4; ++j4) {
                        const f32x4_t av = *reinterpret_cast<const f32x4_t *>(few_lds + t * I + k + j4 * 4);
#pragma unroll
                        for (int j = 0; j < 4; ++j) d = __builtin_fmaf(f[j4 * 4 + j], av[j], d);
                    }
                    // half of one 32-block, its two scales as one exponent (as in gate/up)
                    acc[t][r] += __builtin_ldexpf(d, (int)(we[r] + as[t * (I / 32) + k / 32]) - 254);
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < kRowsPerGroup; ++r) {
            float s = sum_group(acc[t][r], a.lanes);
            if (l == 0 && t < rows && n0 + r < a.H) {
                const int64_t o = (int64_t)t * a.H + n0 + r;
                if (a.addend) s += bf16_to_f32(a.addend[o]);
                a.out[o] = (uint16_t)f32_to_bf16(s);
            }
        }
}

template <class F>
void with_rows(int T, F &&f) {
    if (T == 1) f(std::integral_constant<int, 1>{});
    else f(std::integral_constant<int, kFewRows>{});
}

// The largest power of two of lanes that a row of K values keeps busy with 16 values each.
int lanes_for(int K) {
    int l = 64;
    while (l * 16 > K) l /= 2;
    return l;
}

}  // namespace

hipError_t ffn_few_forward(const FfnPlan &p, char *ws, const uint16_t *x, const mok_weights &w, const uint16_t *addend,
                           uint16_t *out, uint16_t *h, hipStream_t st) {
    const FewArgs a{p.H, p.I, p.few_runs, p.few_run_rows, x, static_cast<const uint16_t *>(w.w_gate),
                    static_cast<const uint16_t *>(w.w_up), static_cast<const uint16_t *>(w.w_down), addend, out, h,
                    reinterpret_cast<float *>(ws + p.part)};
    const int rows = (int)p.T;
    with_rows(rows, [&](auto tc) {
        constexpr int T = decltype(tc)::value;
        {
            KernelTimer tm("ffn_few_gate_up", st);
            const size_t lds = sizeof(float) * T * (p.few_run_rows + kWaves * 128);
            few_gate_up<T><<<(unsigned)(p.I / 64 * p.few_runs), kThreads, lds, st>>>(a, rows);
        }
        KernelTimer tm("ffn_few_down", st);
        const unsigned grid = (unsigned)(ceil_div(p.H / 32, 2 * kXcds) * 2 * kXcds);
        few_down<T><<<grid, kThreads, sizeof(float) * T * (p.I + kWaves * 32), st>>>(a, rows);
    });
    return hipGetLastError();
}

hipError_t ffn_few_mx_forward(const FfnPlan &p, char *ws, const uint8_t *x_elems, const uint8_t *x_scales,
                              const mok_weights &w, const uint16_t *addend, uint16_t *out, uint16_t *h,
                              hipStream_t st) {
    Few8Args a{p.H, p.I, lanes_for(p.H), x_elems, x_scales, w.gate_elems, w.gate_scales, w.up_elems, w.up_scales,
               w.down_elems, w.down_scales, addend, out, h, reinterpret_cast<float *>(ws + p.part)};
    const int rows = (int)p.T;
    with_rows(rows, [&](auto tc) {
        constexpr int T = decltype(tc)::value;
        {
            KernelTimer tm("ffn_few_gate_up_mx", st);
            few_gate_up8<T><<<(unsigned)ceil_div(p.I, kWaves * (64 / a.lanes)), kThreads, 0, st>>>(a, rows);
        }
        a.lanes = lanes_for(p.I);
        KernelTimer tm("ffn_few_down_mx", st);
        const unsigned grid = (unsigned)ceil_div(p.H, kWaves * (64 / a.lanes) * kRowsPerGroup);
        few_down8<T><<<grid, kThreads, sizeof(float) * T * (p.I + p.I / 32), st>>>(a, rows);
    });
    return hipGetLastError();
}

}  // namespace mok
