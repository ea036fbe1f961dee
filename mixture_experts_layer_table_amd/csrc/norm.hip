// Residual addition (with dropout of the added branch) and root-mean-square
// norm, forward and backward.
//   s    = residual + keep * x / (1 - p)          (fp32; stored as the stream's type)
//   rstd = 1 / sqrt(mean_h s^2 + eps)
//   y    = s * rstd * weight                       (bf16 rows, MXFP8 rows, or both)
// Backward, from the stored s, rstd, the weight, dy and the gradient dsum that
// reaches s along the residual stream:
//   g   = dy * weight,  c = rstd^2 * mean_h(g s)
//   ds  = dsum + rstd * (g - s c)                  (the residual's gradient)
//   dx  = keep * ds / (1 - p)
//   dweight_h = sum_t dy s rstd
// The statistics and y are taken from the fp32 sum, before it is rounded to
// the stream's type; the MXFP8 elements are rounded from the fp32 y, not from
// its bf16 copy: one rounding each.
//
// One workgroup per row, the row in registers: one pass over memory, bound by
// HBM. A thread holds CH chunks of 8 elements, chunk c = i * threads + thread, so
// that 4 neighbouring lanes hold one 32-value MXFP8 block. Measured: forward
// 16,384 x 7,168 with dropout, bf16 and MXFP8 rows out, 185 us for 1.06 GB
// (5.7 TB/s; a large copy moves 5.2), 2,048 x 7,168 in fp32 41 us (4.7 TB/s), one
// row 2.6 us; backward 16,384 x 7,168 181 us for 940 MB (5.2 TB/s), 777 x 4,096 in
// fp32 with dropout 16 us (3.3 TB/s: two short kernels).
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "lanes.h"
#include "mx_codec.h"
#include "rng.h"
#include "timing.h"

namespace mok {
namespace {

constexpr int kMaxWaves = 16;

// Sum over the workgroup in a fixed order; `red` holds one float per wave. One
// barrier: a caller that sums twice alternates between two buffers, so a wave
// that runs ahead never overwrites what another still reads.
__device__ __forceinline__ float block_sum(float x, float *red) {
    const int nw = (int)(blockDim.x >> 6), wave = (int)(threadIdx.x >> 6);
    x = sum_wave(x);
    if (nw == 1) return x;
    if ((threadIdx.x & 63) == 0) red[wave] = x;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < nw; ++w) s += red[w];
    return s;
}

struct NormFwdArgs {
    const uint16_t *x;
    const void *residual;
    const uint16_t *weight;
    void *sum;
    uint16_t *y;
    uint8_t *elems, *scales;
    float *rstd;
    DropArgs drop;
    float eps;
    int H;
    int64_t row0;   // first row of the launch
};

template <Elem RES, Elem SUM, int CH>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_forward(NormFwdArgs a) {
    __shared__ float red[kMaxWaves];
    const int64_t row = a.row0 + blockIdx.x;
    const int nc = a.H / 8, nt = (int)blockDim.x, tid = (int)threadIdx.x;
    const int64_t base = row * nc;   // in chunks
    Raw8<kBf16> xr[CH], wr[CH];
    Raw8<RES> rr[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * nt + tid;
        if (c < nc) {
            xr[i] = load8<kBf16>(a.x, base + c);
            rr[i] = load8<RES>(a.residual, base + c);
        }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * nt + tid;
        if (c < nc) wr[i] = load8<kBf16>(a.weight, c);
    }
    const bool drop = a.drop.rng != nullptr;
    const DropState st = drop ? drop_state(a.drop.rng) : DropState{};
    float v[CH][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * nt + tid;
        if (c < nc) {
            float f[8];
            unpack8(xr[i], f);
            unpack8(rr[i], v[i]);
            if (drop) {
                const Words8 w = drop_words8(st, base + c);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = drop_add(f[j], w.w[j], a.drop, v[i][j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += f[j];
            }
            if (a.sum) store8<SUM>(a.sum, base + c, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(v[i][j], v[i][j], ss);
    }
    // a division: 1 / H as a factor would carry its own rounding into every row
    const float r = 1.0f / sqrtf(block_sum(ss, red) / (float)a.H + a.eps);
    if (tid == 0) a.rstd[row] = r;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * nt + tid;
        const bool ok = c < nc;
        float w[8];
        unpack8(wr[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = ok ? v[i][j] * r * w[j] : 0.0f;
        if (a.y && ok) store8<kBf16>(a.y, base + c, v[i]);
        if (a.elems) {   // the same for every thread: the shuffles below see whole waves
            uint32_t amax = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
            amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));   // the 4 lanes of a 32-block
            amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
            const uint32_t sb = mx_scale_byte_f32(amax);
            const uint32_t nan = mx_nan_f32(amax);
            const float q = mx_pow2_neg((int)sb - 127);
            auto codes = [&](int j) {
                return nan | e4m3x2_scaled(v[i][j] * q, v[i][j + 1] * q) |
                       (e4m3x2_scaled(v[i][j + 2] * q, v[i][j + 3] * q) << 16);
            };
            if (ok) {
                reinterpret_cast<uint2 *>(a.elems)[base + c] = make_uint2(codes(0), codes(4));
                if ((c & 3) == 0) a.scales[(base + c) >> 2] = (uint8_t)sb;
            }
        }
    }
}

struct NormBwdArgs {
    const uint16_t *dy;
    const void *sum, *dsum;
    const uint16_t *weight;
    const float *rstd;
    void *dres;
    uint16_t *dx;
    float *part;   // [workgroups][H]: each workgroup's share of dweight
    DropArgs drop;
    int H;
    int64_t T;
};

// Workgroup b walks rows b, b + grid, ...; its dweight share stays in registers.
template <Elem SUM, int CH>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_backward(NormBwdArgs a) {
    __shared__ float red[2][kMaxWaves];
    const int nc = a.H / 8, nt = (int)blockDim.x, tid = (int)threadIdx.x;
    const bool drop = a.drop.rng != nullptr;
    const DropState st = drop ? drop_state(a.drop.rng) : DropState{};
    Raw8<kBf16> wr[CH];
    float dw[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * nt + tid;
        wr[i] = Raw8<kBf16>{make_uint4(0, 0, 0, 0)};
        if (c < nc) wr[i] = load8<kBf16>(a.weight, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        const int64_t base = row * nc;
        Raw8<SUM> sr[CH], er[CH];
        Raw8<kBf16> gr[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + tid;
            if (c < nc) {
                sr[i] = load8<SUM>(a.sum, base + c);
                gr[i] = load8<kBf16>(a.dy, base + c);
                if (a.dsum) er[i] = load8<SUM>(a.dsum, base + c);
            }
        }
        const float r = a.rstd[row];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + tid;
            if (c < nc) {
                float s[8], g[8], w[8];
                unpack8(sr[i], s);
                unpack8(gr[i], g);
                unpack8(wr[i], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dot = __builtin_fmaf(g[j] * w[j], s[j], dot);
                    dw[i][j] = __builtin_fmaf(g[j], s[j] * r, dw[i][j]);
                }
            }
        }
        const float cr = block_sum(dot, red[turn]) / (float)a.H * r * r;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + tid;
            if (c < nc) {
                float s[8], g[8], w[8], d[8];
                unpack8(sr[i], s);
                unpack8(gr[i], g);
                unpack8(wr[i], w);
                if (a.dsum) {
                    unpack8(er[i], d);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = __builtin_fmaf(r, g[j] * w[j] - s[j] * cr, d[j]);
                if (a.dres) store8<SUM>(a.dres, base + c, d);
                if (a.dx) {
                    if (drop) {
                        const Words8 k = drop_words8(st, base + c);
#pragma unroll
                        for (int j = 0; j < 8; ++j) d[j] = drop_add(d[j], k.w[j], a.drop, 0.0f);
                    }
                    store8<kBf16>(a.dx, base + c, d);
                }
            }
        }
    }
    float *part = a.part + (int64_t)blockIdx.x * a.H;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * nt + tid;
        if (c < nc) store8<kF32>(part, c, dw[i]);
    }
}

// dweight[h] = sum over the workgroups' shares: kGroups threads of a column
// each add every kGroups-th share in ascending order, then the groups in order.
constexpr int kCols = 32, kGroups = 16;
__global__ __launch_bounds__(kCols *kGroups) void norm_dweight(const float *__restrict__ part, int n, int H,
                                                               float *__restrict__ dweight) {
    __shared__ float red[kGroups][kCols];
    const int col = threadIdx.x % kCols, grp = threadIdx.x / kCols;
    const int h = blockIdx.x * kCols + col;
    float s = 0.0f;
    if (h < H) {
        for (int i0 = grp; i0 < n; i0 += 8 * kGroups) {   // 8 loads in flight
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = part[(int64_t)min(i0 + j * kGroups, n - 1) * H + h];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i0 + j * kGroups < n) s += v[j];
        }
    }
    red[grp][col] = s;
    __syncthreads();
    if (grp == 0 && h < H) {
        for (int g = 1; g < kGroups; ++g) s += red[g][col];
        dweight[h] = s;
    }
}

// Chunks per thread and waves per workgroup for rows of H elements. One chunk a
// thread up to 8 waves, and for few rows at any width (one row of 7,168: 3.5
// against 3.7 us); past 8 waves two chunks a thread keep more rows in flight on
// a compute unit (16,384 x 7,168 forward: 184 us against 192).
struct RowShape {
    int ch, waves;
};
RowShape row_shape(int H, int64_t rows) {
    const int nc = (H + 7) / 8, one = (nc + 63) / 64, two = (nc + 127) / 128;
    if (one <= 8 || (rows <= 1024 && one <= kMaxWaves)) return RowShape{1, one};
    return RowShape{2, two};   // H <= kNormMaxH
}

// Workgroups of the backward: about kBwdWaves waves in all, each with an equal
// number of rows. More shares cost their traffic (16,384 x 7,168: 182 us with
// 432 workgroups, 192 with 1,024), fewer leave units idle (16,384 x 512: 55 us
// with 256, 23 with 1,024).
constexpr int kBwdWaves = 3000;
int backward_target(int H, int64_t T) { return std::max(1, kBwdWaves / row_shape(H, T).waves); }

template <class F>
void with_ch(int ch, F &&f) {
    if (ch == 1) f(std::integral_constant<int, 1>{});
    else f(std::integral_constant<int, 2>{});
}

}  // namespace

int norm_backward_blocks(int64_t T, int H) {
    const int64_t target = backward_target(H, T), rows = std::max<int64_t>(1, (T + target / 2) / target);
    return (int)((T + rows - 1) / rows);
}

// Shares that a workspace for T rows holds: at least those of every smaller T
// (at most 1.5 times the target, whichever row shape they take).
int64_t norm_backward_shares(int64_t T, int H) {
    return std::min<int64_t>(T, 2 * std::max(backward_target(H, 1), backward_target(H, 1 << 20)));
}

// Threads of one forward launch: a grid takes fewer than 2^32, so rows past that
// many waves (2^25 rows at the narrowest) go to further launches.
constexpr int64_t kLaunchThreads = int64_t(1) << 31;

mok_status launch_add_rmsnorm(const NormCall &c, hipStream_t st) {
    NormFwdArgs a{c.x,  c.residual, c.weight, c.sum, c.y, c.elems, c.scales, c.rstd, drop_args(c.p, c.rng),
                        c.eps, c.H, 0};
    const RowShape rs = row_shape(c.H, c.T);
    const int64_t rows = kLaunchThreads / (64 * rs.waves);
    with_ch(rs.ch, [&](auto ch) {
        constexpr int CH = decltype(ch)::value;
        for (; a.row0 < c.T; a.row0 += rows) {
            const dim3 g((unsigned)std::min(rows, c.T - a.row0)), b(64 * rs.waves);
            KernelTimer tm("add_rmsnorm", st);
            if (c.f32_stream) {
                if (c.residual) norm_forward<kF32, kF32, CH><<<g, b, 0, st>>>(a);
                else norm_forward<kNone, kF32, CH><<<g, b, 0, st>>>(a);
            } else {
                if (c.residual) norm_forward<kBf16, kBf16, CH><<<g, b, 0, st>>>(a);
                else norm_forward<kNone, kBf16, CH><<<g, b, 0, st>>>(a);
            }
        }
    });
    return check_hip(hipGetLastError(), "mok_add_rmsnorm");
}

mok_status launch_add_rmsnorm_backward(const NormBackwardCall &c, hipStream_t st) {
    const NormBwdArgs a{c.dy,  c.sum, c.dsum, c.weight, c.rstd, c.dres, c.dx, c.part, drop_args(c.p, c.rng),
                        c.H, c.T};
    const int blocks = norm_backward_blocks(c.T, c.H);
    const RowShape rs = row_shape(c.H, c.T);
    if (blocks > 0) {
        KernelTimer tm("add_rmsnorm_backward", st);
        with_ch(rs.ch, [&](auto ch) {
            constexpr int CH = decltype(ch)::value;
            if (c.f32_stream) norm_backward<kF32, CH><<<blocks, 64 * rs.waves, 0, st>>>(a);
            else norm_backward<kBf16, CH><<<blocks, 64 * rs.waves, 0, st>>>(a);
        });
    }
    {
        KernelTimer tm("norm_dweight", st);
        norm_dweight<<<(unsigned)((c.H + kCols - 1) / kCols), kCols * kGroups, 0, st>>>(c.part, blocks, c.H, c.dweight);
    }
    return check_hip(hipGetLastError(), "mok_add_rmsnorm_backward");
}

}  // namespace mok
