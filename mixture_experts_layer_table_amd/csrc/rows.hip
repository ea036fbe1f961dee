// Token rows sorted by expert and back, and both gradients. With slot[t,j] the
// row of token t's j-th choice (below 0: none):
//   permute            rows[slot[t,j]] = x[t]            (as they are, or in 8-bit blocks of 128)
//   unpermute          out[t] = addend[t] + sum_j w[t,j] y[slot[t,j]]
//   permute backward   the same sum without weights
//   unpermute backward dy[slot[t,j]] = w[t,j] dout[t],  dw[t,j] = <dout[t], y[slot[t,j]]>
// All four go by token: a token's row is read once and stays in registers
// while its k rows are written (and quantized once, not k times), or its k rows
// are read into one sum; no row is touched twice and nothing is added through
// memory. Bound by HBM; 2,048 tokens of 7,168 bf16, 8 choices each: permute to 8-bit
// rows 31 us (4.8 TB/s; its scales go out as single words), as they are 53 us (5.5
// TB/s; of fp32 242 us, 2.4 TB/s), unpermute 55 us (5.3 TB/s). Unpermute backward,
// 1,001 x 4,096 fp32, 2 choices: 15.4 us in a stream of calls (4.3 TB/s: 66 MB, of
// which a launch's start and end are a quarter), 16.8 alone.
//
// Rows that pad an expert's run get zeros from workgroups of their own in the
// same launch. Slots are checked against the number of rows, so a damaged table
// can give wrong rows but no access out of range.
#include "fp8_codec.h"
#include "kernels.h"
#include "lanes.h"
#include "stream.h"
#include "timing.h"

namespace mok {
namespace {

constexpr int kRowThreads = 256;            // a chunk of 8 elements each
// Rows that a wave and a workgroup look over for padding. Two a wave: an expert's padding is one run of rows, and a
// wave that fills eight of them ends last (1,001 x 4,096 in fp32, two rows a token, 128-row runs: 22 against 16 us).
constexpr int kPadWave = 2, kPadRows = kPadWave * kRowThreads / 64;
constexpr int kBatch = 8;                   // rows in flight per thread
constexpr int64_t kMostGroups = 1 << 23;    // workgroups of a launch: a grid takes fewer than 2^32 threads

struct RowsArgs {
    RowsCall c;
    const void *x, *y, *addend;
    const float *w;
    void *rows, *out;
    uint8_t *elems;
    float *scales, *dw;
    int64_t first;       // first workgroup of the launch
    int64_t tokens_end;  // workgroups below this one take tokens, the others padding
    int strips;          // workgroups per token
};

__device__ __forceinline__ bool row_ok(const RowsCall &c, int64_t row) { return (uint64_t)row < (uint64_t)c.rows; }

// The rows (or -1) of slots [j0, j0 + N) of token t, read ahead of any store: a load behind one would be made again.
template <int N>
struct SlotRows {
    int r[N];
    __device__ __forceinline__ SlotRows(const RowsCall &c, int64_t t, int j0) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            r[j] = j0 + j < c.k ? c.slots[t * c.k + j0 + j] : -1;
            if (!row_ok(c, r[j])) r[j] = -1;
        }
    }
};

// Zeros into the padding rows among this wave's.
template <Elem E, bool ROWS, bool FP8>
__device__ __forceinline__ void pad_rows(const RowsArgs &a, int64_t group) {
    const RowsCall &c = a.c;
    const int lane = (int)(threadIdx.x & 63), nc = c.H / 8;
    const int64_t r0 = group * kPadRows + (threadIdx.x >> 6) * kPadWave, end = min((int64_t)c.offsets[c.E], c.rows);
    for (int i = 0; i < kPadWave; ++i) {
        const int64_t r = r0 + i;
        if (r >= end) return;
        if (c.row_slots[r] >= 0) continue;
        const float zero[8] = {};
        for (int h = lane; h < nc; h += 64) {
            if constexpr (ROWS) stream8_elems<E>(a.rows, r * nc + h, zero);
            if constexpr (FP8) stream8(a.elems, r * nc + h, make_uint2(0, 0));
        }
        if constexpr (FP8)
            for (int kb = lane; kb < (c.H + kBlk - 1) / kBlk; kb += 64) a.scales[kb * c.rows + r] = kLeastScale;
    }
}

// The row as it is: a chunk of 8 elements a thread.
template <Elem E>
__global__ __launch_bounds__(kRowThreads) void permute_kernel(RowsArgs a) {
    const RowsCall &c = a.c;
    const int64_t b = a.first + blockIdx.x;
    if (b >= a.tokens_end) {
        pad_rows<E, true, false>(a, b - a.tokens_end);
        return;
    }
    const int64_t t = b / a.strips;
    const int nc = c.H / 8, h = (int)(b % a.strips) * kRowThreads + (int)threadIdx.x;
    if (h >= nc) return;
    const Raw8<E> v = load8<E>(a.x, t * nc + h);
    for (int j0 = 0; j0 < c.k; j0 += kBatch) {
        const SlotRows<kBatch> s(c, t, j0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (s.r[j] >= 0) stream8_raw<E>(a.rows, (int64_t)s.r[j] * nc + h, v);
    }
}

// The row quantized (and as it is, with ROWS): 16 elements a thread, 8 neighbouring
// lanes a block. H is a multiple of 16. 16-byte stores of codes instead of 8-byte
// ones: 2,048 x 7,168 to 8 rows each, with non-temporal ones, 44 -> 31 us.
template <Elem E, bool ROWS>
__global__ __launch_bounds__(kRowThreads) void permute_quantized(RowsArgs a) {
    const RowsCall &c = a.c;
    const int64_t b = a.first + blockIdx.x;
    if (b >= a.tokens_end) {
        pad_rows<E, ROWS, true>(a, b - a.tokens_end);
        return;
    }
    const int64_t t = b / a.strips;
    const int nu = c.H / 16, u = (int)(b % a.strips) * kRowThreads + (int)threadIdx.x;
    const bool live = u < nu;
    Raw8<E> lo = {}, hi = {};
    if (live) {
        lo = load8<E>(a.x, (t * nu + u) * 2);
        hi = load8<E>(a.x, (t * nu + u) * 2 + 1);
    }
    float v[8], w[8];
    unpack8(lo, v);
    unpack8(hi, w);
    const BlkScale s = blk_scale(max8(max(amax8(v), amax8(w))));
    const uint4 q = make_uint4(blk_codes4(s, v[0], v[1], v[2], v[3]), blk_codes4(s, v[4], v[5], v[6], v[7]),
                               blk_codes4(s, w[0], w[1], w[2], w[3]), blk_codes4(s, w[4], w[5], w[6], w[7]));
    if (!live) return;
    for (int j0 = 0; j0 < c.k; j0 += kBatch) {
        const SlotRows<kBatch> to(c, t, j0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t r = to.r[j];
            if (r < 0) continue;
            if constexpr (ROWS) {
                stream8_raw<E>(a.rows, (r * nu + u) * 2, lo);
                stream8_raw<E>(a.rows, (r * nu + u) * 2 + 1, hi);
            }
            stream16(a.elems, r * nu + u, q);
            if (u % 8 == 0) a.scales[u / 8 * c.rows + r] = s.scale;
        }
    }
}

template <Elem E, bool W>
__global__ __launch_bounds__(kRowThreads) void unpermute_kernel(RowsArgs a) {
    const RowsCall &c = a.c;
    const int64_t b = a.first + blockIdx.x, t = b / a.strips;
    const int nc = c.H / 8, h = (int)(b % a.strips) * kRowThreads + (int)threadIdx.x;
    if (h >= nc) return;
    float s[8] = {}, add[8] = {};
    if (a.addend) unpack8(load8<E>(a.addend, t * nc + h), add);
    for (int j0 = 0; j0 < c.k; j0 += kBatch) {
        const SlotRows<kBatch> from(c, t, j0);
        Raw8<E> raw[kBatch] = {};
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (from.r[j] >= 0) raw[j] = load8<E>(a.y, (int64_t)from.r[j] * nc + h);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (from.r[j] < 0) continue;   // nothing, whatever its weight
            float v[8], w = 1.0f;
            if constexpr (W) w = a.w[t * c.k + j0 + j];
            unpack8(raw[j], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = __builtin_fmaf(w, v[i], s[i]);
        }
    }
    if (a.addend) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += add[i];
    }
    stream8_elems<E>(a.out, t * nc + h, s);
}

// One workgroup a token, with the partial dots of up to kBatch choices in registers.
// A thread asks for CH chunks of dout and of up to NB choices' rows before it uses
// the first: a row is a few chunks a thread, so a call lives on what is in flight.
template <Elem E, int CH, int NB>
__global__ __launch_bounds__(kRowThreads) void unpermute_backward_kernel(RowsArgs a) {
    __shared__ float red[kRowThreads / 64][NB];
    const RowsCall &c = a.c;
    const int64_t b = a.first + blockIdx.x;
    if (b >= a.tokens_end) {
        pad_rows<E, true, false>(a, b - a.tokens_end);
        return;
    }
    const int64_t t = b;
    const int nc = c.H / 8, tid = (int)threadIdx.x, wave = tid >> 6;
    for (int j0 = 0; j0 < c.k; j0 += NB) {
        const SlotRows<NB> to(c, t, j0);
        float dot[NB] = {}, w[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) w[j] = to.r[j] >= 0 ? a.w[t * c.k + j0 + j] : 0.0f;
        for (int h0 = tid; h0 < nc; h0 += CH * kRowThreads) {
            Raw8<E> dr[CH] = {}, yr[CH][NB] = {};
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int h = h0 + i * kRowThreads;
                if (h < nc) dr[i] = load8<E>(a.x, t * nc + h);
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    if (h < nc && to.r[j] >= 0) yr[i][j] = load8<E>(a.y, (int64_t)to.r[j] * nc + h);
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int h = h0 + i * kRowThreads;
                float d[8];
                unpack8(dr[i], d);
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    if (h >= nc || to.r[j] < 0) continue;
                    float v[8], g[8];
                    unpack8(yr[i][j], v);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        dot[j] = __builtin_fmaf(d[q], v[q], dot[j]);
                        g[q] = w[j] * d[q];
                    }
                    // y's own chunk may lie here: read above, by this thread alone
                    stream8_elems<E>(a.rows, (int64_t)to.r[j] * nc + h, g);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const float s = sum_wave(dot[j]);
            if ((tid & 63) == 0) red[wave][j] = s;
        }
        __syncthreads();
        if (tid < NB && j0 + tid < c.k) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kRowThreads / 64; ++w) s += red[w][tid];
            a.dw[t * c.k + j0 + tid] = s;   // 0 for a slot without a row
        }
        __syncthreads();
    }
}

template <class K>
hipError_t launch_groups(K kernel, const char *name, RowsArgs a, int64_t groups, hipStream_t st) {
    KernelTimer tm(name, st);
    for (a.first = 0; a.first < groups; a.first += kMostGroups) {
        const int64_t n = groups - a.first < kMostGroups ? groups - a.first : kMostGroups;
        kernel<<<(unsigned)n, kRowThreads, 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

int64_t ceil_of(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

mok_status launch_permute(const RowsCall &c, const void *x, void *rows, uint8_t *elems, float *scales,
                          hipStream_t st) {
    RowsArgs a{};
    a.c = c;
    a.x = x;
    a.rows = rows;
    a.elems = elems;
    a.scales = scales;
    a.strips = (int)ceil_of(c.H / (elems ? 16 : 8), kRowThreads);
    a.tokens_end = c.T * a.strips;
    const int64_t groups = a.tokens_end + ceil_of(c.rows, kPadRows);
    hipError_t e;
    if (elems) {
        if (c.f32)
            e = rows ? launch_groups(permute_quantized<kF32, true>, "permute", a, groups, st)
                     : launch_groups(permute_quantized<kF32, false>, "permute", a, groups, st);
        else
            e = rows ? launch_groups(permute_quantized<kBf16, true>, "permute", a, groups, st)
                     : launch_groups(permute_quantized<kBf16, false>, "permute", a, groups, st);
    } else {
        e = c.f32 ? launch_groups(permute_kernel<kF32>, "permute", a, groups, st)
                  : launch_groups(permute_kernel<kBf16>, "permute", a, groups, st);
    }
    return check_hip(e, "mok_permute");
}

mok_status launch_unpermute(const RowsCall &c, const void *y, const float *w, const void *addend, void *out,
                            const char *where, hipStream_t st) {
    RowsArgs a{};
    a.c = c;
    a.y = y;
    a.w = w;
    a.addend = addend;
    a.out = out;
    a.strips = (int)ceil_of(c.H / 8, kRowThreads);
    const int64_t groups = c.T * a.strips;
    const char *name = "unpermute";
    const hipError_t e = c.f32 ? (w ? launch_groups(unpermute_kernel<kF32, true>, name, a, groups, st)
                                    : launch_groups(unpermute_kernel<kF32, false>, name, a, groups, st))
                               : (w ? launch_groups(unpermute_kernel<kBf16, true>, name, a, groups, st)
                                    : launch_groups(unpermute_kernel<kBf16, false>, name, a, groups, st));
    return check_hip(e, where);
}

mok_status launch_unpermute_backward(const RowsCall &c, const void *dout, const void *y, const float *w, void *dy,
                                     float *dw, hipStream_t st) {
    RowsArgs a{};
    a.c = c;
    a.x = dout;
    a.y = y;
    a.w = w;
    a.rows = dy;
    a.dw = dw;
    a.strips = 1;
    a.tokens_end = c.T;
    const int64_t groups = c.T + ceil_of(c.rows, kPadRows);
    const char *name = "unpermute_backward";
    // Choices at once: two for k <= 2 (1,001 x 4,096 bf16, k = 1: 4.4 us against 5.9 with eight), else eight
    // (1,001 x 4,096 fp32, k = 8: 59 against 62).
    hipError_t e;
    if (c.k <= 2)
        e = c.f32 ? launch_groups(unpermute_backward_kernel<kF32, 2, 2>, name, a, groups, st)
                  : launch_groups(unpermute_backward_kernel<kBf16, 4, 2>, name, a, groups, st);
    else
        e = c.f32 ? launch_groups(unpermute_backward_kernel<kF32, 1, kBatch>, name, a, groups, st)
                  : launch_groups(unpermute_backward_kernel<kBf16, 1, kBatch>, name, a, groups, st);
    return check_hip(e, "mok_unpermute_backward");
}

}  // namespace mok
