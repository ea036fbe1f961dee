// Dropout of a branch, with the residual's addition:
//   out = residual + keep * x / (1 - p)        (forward)
//   dx  = keep * dy / (1 - p)                  (backward: the same kernel without a residual)
// The mask comes from the counter-based generator in rng.h and is never stored.
//
// One pass over the data; a thread takes 16-byte chunks of 8 elements, two
// generator blocks each, with the loads of 4 chunks in flight before the first
// block is computed. Bound by HBM: the 20 wide multiplies of a block take about
// 80 us of vector time at 16,384 x 7,168, under the transfer's. Measured there,
// bf16 residual: 125 us for 705 MB (5.6 TB/s; a large copy moves 5.2); gradient
// of 2,047 x 4,096 in fp32: 9.7 us for 50 MB.
#include "kernels.h"
#include "rng.h"
#include "timing.h"

namespace mok {
namespace {

constexpr int kDropThreads = 256;
constexpr int kDropChunks = 4;   // chunks in flight per thread
static_assert((kMaxDropout + 8191) / 8192 * kDropThreads < int64_t(1) << 32 && kDropThreads * kDropChunks * 8 == 8192,
              "the largest call fits one grid");

template <Elem IN, Elem RES, Elem OUT>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(const void *x, const void *residual,
                                                               int64_t n, DropArgs d, void *out) {
    const int64_t nc = n / 8;
    const int64_t c0 = (int64_t)blockIdx.x * (kDropThreads * kDropChunks) + threadIdx.x;
    const bool drop = d.rng != nullptr;
    const DropState st = drop ? drop_state(d.rng) : DropState{};
    Raw8<IN> xr[kDropChunks];
    Raw8<RES> rr[kDropChunks];
#pragma unroll
    for (int i = 0; i < kDropChunks; ++i) {
        const int64_t c = c0 + i * kDropThreads;
        if (c < nc) {
            xr[i] = load8<IN>(x, c);
            rr[i] = load8<RES>(residual, c);
        }
    }
#pragma unroll
    for (int i = 0; i < kDropChunks; ++i) {
        const int64_t c = c0 + i * kDropThreads;
        if (c >= nc) break;
        float v[8], b[8];
        unpack8(xr[i], v);
        unpack8(rr[i], b);
        if (drop) {
            const Words8 w = drop_words8(st, c);
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = drop_add(v[j], w.w[j], d, b[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] += v[j];
        }
        store8<OUT>(out, c, b);
    }
    // the last n % 8 elements, one thread each, in the first workgroup
    if (blockIdx.x == 0 && threadIdx.x < (unsigned)(n % 8)) {
        const int64_t e = nc * 8 + threadIdx.x;
        auto one = [&](const void *p, Elem k) {
            return k == kF32 ? static_cast<const float *>(p)[e]
                             : __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[e] << 16);
        };
        const float v = one(x, IN);
        float b = 0.0f;
        if constexpr (RES != kNone) b = one(residual, RES);
        if (drop) {
            const uint4 w = philox4x32_10(st.offset + (uint64_t)(e / 4), st.k0, st.k1);
            const uint32_t word = (e & 3) == 0 ? w.x : (e & 3) == 1 ? w.y : (e & 3) == 2 ? w.z : w.w;
            b = drop_add(v, word, d, b);
        } else {
            b += v;
        }
        if constexpr (OUT == kF32)
            static_cast<float *>(out)[e] = b;
        else
            static_cast<uint16_t *>(out)[e] = (uint16_t)f32_to_bf16(b);
    }
}

template <Elem IN, Elem RES, Elem OUT>
hipError_t launch(const char *name, const void *x, const void *residual, int64_t n, const DropArgs &d, void *out,
                  hipStream_t st) {
    const int64_t per = (int64_t)kDropThreads * kDropChunks * 8;
    const int64_t blocks = n < 8 ? 1 : (n / 8 * 8 + per - 1) / per;
    KernelTimer tm(name, st);
    dropout_kernel<IN, RES, OUT><<<(unsigned)blocks, kDropThreads, 0, st>>>(x, residual, n, d, out);
    return hipGetLastError();
}

}  // namespace

mok_status launch_dropout(const uint16_t *x, const void *residual, int64_t n, float p, const uint64_t *rng,
                          bool f32_stream, void *out, hipStream_t st) {
    const DropArgs d = drop_args(p, rng);
    hipError_t e;
    if (f32_stream)
        e = residual ? launch<kBf16, kF32, kF32>("dropout", x, residual, n, d, out, st)
                     : launch<kBf16, kNone, kF32>("dropout", x, residual, n, d, out, st);
    else
        e = residual ? launch<kBf16, kBf16, kBf16>("dropout", x, residual, n, d, out, st)
                     : launch<kBf16, kNone, kBf16>("dropout", x, residual, n, d, out, st);
    return check_hip(e, "mok_dropout");
}

mok_status launch_dropout_backward(const void *dy, int64_t n, float p, const uint64_t *rng, bool f32_stream,
                                   uint16_t *dx, hipStream_t st) {
    const DropArgs d = drop_args(p, rng);
    const hipError_t e = f32_stream ? launch<kF32, kNone, kBf16>("dropout_backward", dy, nullptr, n, d, dx, st)
                                    : launch<kBf16, kNone, kBf16>("dropout_backward", dy, nullptr, n, d, dx, st);
    return check_hip(e, "mok_dropout_backward");
}

}  // namespace mok
