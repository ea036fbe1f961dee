// Quantization into blocks of 128 with one fp32 scale (fp8_codec.h), and the
// gradient of the gated activation. One pass over the data: a block's values
// stay in registers between its largest magnitude and its codes. Bound by HBM.
//
//   rows    src [rows][K]: 16 neighbouring lanes hold a block, 8 values each; a
//           workgroup takes 16 rows x kRun blocks, so that a block's 16 scales
//           leave as one line of the block-by-block scales.
//   tile    src [rows][K] in 128 x 128 blocks: a workgroup takes one block.
//   turned  src [K][rows], the transpose is quantized: a workgroup takes 128
//           values of K x 128 rows, a thread 8 rows of 8 consecutive k, so that it
//           packs 8 codes of a row at once; they pass through LDS and leave as
//           whole 128-byte lines of their rows.
// Measured: 4 x 4,096 x 7,168 bf16 in tiles 65 us (5.4 TB/s), turned 66 us; 16,384 x 7,168
// rows 62 us (5.7 TB/s), turned 78 (4.6); 16,384 x 2,048 gated rows 33 us (5.2 TB/s), turned
// 35; 2,047 x 2,048 gated rows 6.5 us alone (3.2 TB/s: 21 MB are a short launch); the
// gated activation's gradient of 16,384 x 2,048 57 us (5.9 TB/s).
// With GLU the source rows are [g | u] and v = silu(g) * u is quantized.
#include "fp8_codec.h"
#include "glu.h"
#include "kernels.h"
#include "stream.h"
#include "timing.h"

namespace mok {
namespace {

constexpr int kQThreads = 256;
constexpr int kRun = 2;                     // blocks of a row per thread (16,384 x 7,168: 1, 2, 4 blocks 69, 62, 65 us)
constexpr int64_t kMostGroups = 1 << 23;    // workgroups of a launch: a grid takes fewer than 2^32 threads

struct QuantArgs {
    const void *src;
    uint8_t *elems;
    float *scales;
    int64_t rows, K, kblocks;   // of one matrix
    int64_t per, cols;          // workgroups of a matrix, and of one row of them
    int64_t first;              // first workgroup of the launch
};

// 8 values from chunk c (of 8 elements); GLU: u lies `half` chunks further.
template <Elem E, bool GLU>
struct Source8 {
    Raw8<E> g, u;
    __device__ __forceinline__ void load(const void *src, int64_t c, int64_t half) {
        g = load8<E>(src, c);
        if constexpr (GLU) u = load8<E>(src, c + half);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        unpack8(g, v);
        if constexpr (GLU) {
            float w[8];
            unpack8(u, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = glu_forward(v[j], w[j]);
        }
    }
};

template <Elem E, bool GLU>
__global__ __launch_bounds__(kQThreads) void quantize_rows(QuantArgs a) {
    const int64_t b = a.first + blockIdx.x, m = b / a.per, o = b % a.per;
    const int lane = (int)threadIdx.x & 15;
    const int64_t r = o / a.cols * 16 + (threadIdx.x >> 4), kb0 = o % a.cols * kRun, nc = a.K / 8;
    const bool row = r < a.rows;   // whole groups of 16 lanes
    const int64_t src_row = (m * a.rows + (row ? r : 0)) * nc * (GLU ? 2 : 1), dst_row = (m * a.rows + r) * nc;
    Source8<E, GLU> s[kRun] = {};
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        const int64_t c = (kb0 + i) * 16 + lane;
        if (row && c < nc) s[i].load(a.src, src_row + c, nc);
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        const int64_t c = (kb0 + i) * 16 + lane;
        float v[8];
        s[i].values(v);   // zeros behind the row's end
        const BlkScale q = blk_scale(max16(amax8(v)));
        if (!row || c >= nc) continue;
        stream8(a.elems, dst_row + c,
                make_uint2(blk_codes4(q, v[0], v[1], v[2], v[3]), blk_codes4(q, v[4], v[5], v[6], v[7])));
        if (lane == 0) a.scales[(m * a.kblocks + kb0 + i) * a.rows + r] = q.scale;
    }
}

// Largest of the workgroup's values; every thread takes part.
__device__ __forceinline__ uint32_t max_group(uint32_t x, uint32_t *red) {
    x = max16(x);
    x = max(x, (uint32_t)__shfl_xor((int)x, 16));
    x = max(x, (uint32_t)__shfl_xor((int)x, 32));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    for (int w = 0; w < kQThreads / 64; ++w) x = max(x, red[w]);
    return x;
}

template <Elem E>
__global__ __launch_bounds__(kQThreads) void quantize_tiles(QuantArgs a) {
    __shared__ uint32_t red[kQThreads / 64];
    const int64_t b = a.first + blockIdx.x, m = b / a.per, o = b % a.per;
    const int64_t rb = o / a.cols, kb = o % a.cols, nc = a.K / 8;
    const int64_t r0 = rb * kBlk + (threadIdx.x >> 4), c = kb * 16 + (threadIdx.x & 15);
    Raw8<E> raw[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (r0 + i * 16 < a.rows && c < nc) raw[i] = load8<E>(a.src, (m * a.rows + r0 + i * 16) * nc + c);
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        unpack8(raw[i], v);
        amax = max(amax, amax8(v));
    }
    const BlkScale q = blk_scale(max_group(amax, red));
    if (threadIdx.x == 0) a.scales[(m * (a.per / a.cols) + rb) * a.cols + kb] = q.scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        unpack8(raw[i], v);
        if (r0 + i * 16 < a.rows && c < nc)
            stream8(a.elems, (m * a.rows + r0 + i * 16) * nc + c,
                    make_uint2(blk_codes4(q, v[0], v[1], v[2], v[3]), blk_codes4(q, v[4], v[5], v[6], v[7])));
    }
}

// LDS rows of codes: 128 bytes of a row's k and 8 more, so that the 16 lanes
// that write one 8-byte unit of 8 rows each fall on different banks.
constexpr int kTurnRow = kBlk + 8;

template <Elem E, bool TILE, bool GLU>
__global__ __launch_bounds__(kQThreads) void quantize_turned(QuantArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t codes[kBlk * kTurnRow];
    __shared__ uint32_t part[16][kBlk + 4];
    const int64_t b = a.first + blockIdx.x, m = b / a.per, o = b % a.per;
    const int64_t rb = o % a.cols, kb = o / a.cols;          // neighbouring workgroups read neighbouring rows of src
    const int rc = (int)threadIdx.x & 15, kk = (int)threadIdx.x >> 4;
    const int64_t nc = a.rows / 8, c = rb * 16 + rc, k0 = kb * kBlk + kk * 8;
    Source8<E, GLU> s[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k0 + i < a.K && c < nc) s[i].load(a.src, (m * a.K + k0 + i) * nc * (GLU ? 2 : 1) + c, nc);
    float v[8][8];   // [k][row]
    uint32_t amax[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        s[i].values(v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax[j] = max(amax[j], abs_bits(v[i][j]));
    }
    BlkScale q[8];
    if constexpr (TILE) {
        uint32_t x = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) x = max(x, amax[j]);
        const BlkScale one = blk_scale(max_group(x, part[0]));
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = one;
        if (threadIdx.x == 0) a.scales[(m * a.cols + rb) * a.kblocks + kb] = one.scale;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) part[kk][rc * 8 + j] = amax[j];
        __syncthreads();
        if (threadIdx.x < kBlk) {
            uint32_t x = 0;
#pragma unroll
            for (int g = 0; g < 16; ++g) x = max(x, part[g][threadIdx.x]);
            part[0][threadIdx.x] = x;   // read above by this thread alone
            const int64_t r = rb * kBlk + threadIdx.x;
            if (r < a.rows) a.scales[(m * a.kblocks + kb) * a.rows + r] = blk_scale(x).scale;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = blk_scale(part[0][rc * 8 + j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint2 *>(codes + (rc * 8 + j) * kTurnRow + kk * 8) =
            make_uint2(blk_codes4(q[j], v[0][j], v[1][j], v[2][j], v[3][j]),
                       blk_codes4(q[j], v[4][j], v[5][j], v[6][j], v[7][j]));
    __syncthreads();
    // 8 lanes a row, 16 bytes each: K is a multiple of 16
    const int unit = (int)threadIdx.x & 7;
    const int64_t k = kb * kBlk + unit * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int lr = i * 32 + ((int)threadIdx.x >> 3);
        const int64_t r = rb * kBlk + lr;
        if (r >= a.rows || k >= a.K) continue;
        const uint2 lo = *reinterpret_cast<const uint2 *>(codes + lr * kTurnRow + unit * 16);
        const uint2 hi = *reinterpret_cast<const uint2 *>(codes + lr * kTurnRow + unit * 16 + 8);
        stream16(a.elems, ((m * a.rows + r) * a.K + k) / 16, make_uint4(lo.x, lo.y, hi.x, hi.y));
    }
}

template <class K>
hipError_t launch_groups(K kernel, const char *name, QuantArgs a, int64_t groups, hipStream_t st) {
    KernelTimer tm(name, st);
    for (a.first = 0; a.first < groups; a.first += kMostGroups) {
        const int64_t n = groups - a.first < kMostGroups ? groups - a.first : kMostGroups;
        kernel<<<(unsigned)n, kQThreads, 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

int64_t ceil_of(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A thread takes 8 values; da and dh's halves lie in different rows.
__global__ __launch_bounds__(kQThreads) void glu_backward_kernel(const uint16_t *da, const uint16_t *h, int64_t n,
                                                                 int nc, int64_t first, uint16_t *dh) {
    const int64_t c = (first + blockIdx.x) * kQThreads + threadIdx.x;   // chunk of da
    if (c >= n) return;
    const int64_t g = c / nc * nc + c, u = g + nc;   // row t of h begins 2 t nc chunks in: t nc more than da's
    float d[8], hg[8], hu[8];
    const Raw8<kBf16> rd = load8<kBf16>(da, c), rg = load8<kBf16>(h, g), ru = load8<kBf16>(h, u);
    unpack8(rd, d);
    unpack8(rg, hg);
    unpack8(ru, hu);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const GluGrad r = glu_backward(d[j], hg[j], hu[j]);
        hg[j] = r.dg;
        hu[j] = r.du;
    }
    stream8_elems<kBf16>(dh, g, hg);
    stream8_elems<kBf16>(dh, u, hu);
}

}  // namespace

mok_status launch_fp8_quantize(const void *src, bool f32, int64_t batch, int64_t rows, int64_t K, uint32_t flags,
                               uint8_t *elems, float *scales, hipStream_t st) {
    QuantArgs a{};
    a.src = src;
    a.elems = elems;
    a.scales = scales;
    a.rows = rows;
    a.K = K;
    a.kblocks = ceil_of(K, kBlk);
    const bool tile = flags & MOK_FP8_TILE, glu = flags & MOK_FP8_GLU;
    const char *name = "fp8_quantize";
    hipError_t e;
    if (flags & MOK_FP8_TURNED) {
        a.cols = ceil_of(rows, kBlk);
        a.per = a.cols * a.kblocks;
        const int64_t n = batch * a.per;
        if (glu)
            e = launch_groups(quantize_turned<kBf16, false, true>, name, a, n, st);
        else if (f32)
            e = tile ? launch_groups(quantize_turned<kF32, true, false>, name, a, n, st)
                     : launch_groups(quantize_turned<kF32, false, false>, name, a, n, st);
        else
            e = tile ? launch_groups(quantize_turned<kBf16, true, false>, name, a, n, st)
                     : launch_groups(quantize_turned<kBf16, false, false>, name, a, n, st);
    } else if (tile) {
        a.cols = a.kblocks;
        a.per = a.cols * ceil_of(rows, kBlk);
        const int64_t n = batch * a.per;
        e = f32 ? launch_groups(quantize_tiles<kF32>, name, a, n, st)
                : launch_groups(quantize_tiles<kBf16>, name, a, n, st);
    } else {
        a.cols = ceil_of(a.kblocks, kRun);
        a.per = a.cols * ceil_of(rows, 16);
        const int64_t n = batch * a.per;
        e = glu   ? launch_groups(quantize_rows<kBf16, true>, name, a, n, st)
            : f32 ? launch_groups(quantize_rows<kF32, false>, name, a, n, st)
                  : launch_groups(quantize_rows<kBf16, false>, name, a, n, st);
    }
    return check_hip(e, "mok_fp8_quantize");
}

mok_status launch_glu_backward(const uint16_t *da, const uint16_t *h, int64_t T, int I, uint16_t *dh, hipStream_t st) {
    const int nc = I / 8;
    const int64_t n = T * nc, groups = ceil_of(n, kQThreads);
    KernelTimer tm("glu_backward", st);
    for (int64_t first = 0; first < groups; first += kMostGroups) {
        const int64_t g = groups - first < kMostGroups ? groups - first : kMostGroups;
        glu_backward_kernel<<<(unsigned)g, kQThreads, 0, st>>>(da, h, n, nc, first, dh);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return check_hip(e, "mok_glu_backward");
    }
    return MOK_OK;
}

}  // namespace mok
