// Host-side launchers of the device code (one per C-ABI entry point).
#pragma once
#include <hip/hip_runtime.h>

#include "plan.h"

namespace mok {

// Records `err` (with the call site) as the calling thread's last error when it
// is not hipSuccess, and maps it to a status.
mok_status check_hip(hipError_t err, const char *where);
// Sets the calling thread's mok_last_error text.
void set_last_error(const char *text);

mok_status launch_build_schedule(const Plan &p, const int32_t *ids, void *schedule, hipStream_t st);

// Enqueues the fingerprint check of a schedule table against the plan of the
// call that is about to read it (sets MOK_SCHEDULE_MISMATCH on a mismatch).
mok_status launch_schedule_check(const Plan &p, const void *schedule, hipStream_t st);

mok_status launch_forward(const Plan &p, const void *schedule, void *workspace, const uint16_t *x,
                          const float *topk_w, const mok_weights &w, uint16_t *out, void *fwd_ctx,
                          hipStream_t st);

mok_status launch_backward(const Plan &p, const void *schedule, void *workspace, const uint16_t *x,
                           const float *topk_w, const mok_weights &w, const void *fwd_ctx,
                           const uint16_t *dy, uint16_t *dx, uint16_t *dw_gate, uint16_t *dw_up,
                           uint16_t *dw_down, float *dtopk_w, hipStream_t st);

mok_status launch_mxfp8_quantize(const uint16_t *src, int64_t batch, int64_t rows, int64_t K,
                                 bool src_is_k_by_rows, uint8_t *elems, uint8_t *scales, hipStream_t st);

mok_status launch_route(const float *logits, int64_t T, int E, int k, int32_t *ids, float *w, hipStream_t st);

mok_status launch_route_backward(const int32_t *ids, const float *w, const float *dw, int64_t T, int E, int k,
                                 float *dl, hipStream_t st);

// Most elements of one dropout call: a grid takes fewer than 2^32 threads, and a
// workgroup of 256 takes 8,192 elements.
constexpr int64_t kMaxDropout = ((int64_t(1) << 24) - 1) * 8192;
mok_status launch_dropout(const uint16_t *x, const void *residual, int64_t n, float p, const uint64_t *rng,
                          bool f32_stream, void *out, hipStream_t st);

mok_status launch_dropout_backward(const void *dy, int64_t n, float p, const uint64_t *rng, bool f32_stream,
                                   uint16_t *dx, hipStream_t st);

constexpr int kNormMaxH = 16384;   // 16 waves x 2 chunks of 8 elements per lane

struct NormCall {
    int64_t T;
    int H;
    float eps, p;
    bool f32_stream;
    const uint16_t *x;
    const void *residual;
    const uint16_t *weight;
    const uint64_t *rng;
    void *sum;
    uint16_t *y;
    uint8_t *elems, *scales;
    float *rstd;
};
mok_status launch_add_rmsnorm(const NormCall &c, hipStream_t st);

struct NormBackwardCall {
    int64_t T;
    int H;
    float p;
    bool f32_stream;
    const uint16_t *dy;
    const void *sum, *dsum;
    const uint16_t *weight;
    const float *rstd;
    const uint64_t *rng;
    void *dres;
    uint16_t *dx;
    float *dweight;
    float *part;   // norm_backward_shares(T, H) x H floats
};
int64_t norm_backward_shares(int64_t T, int H);
mok_status launch_add_rmsnorm_backward(const NormBackwardCall &c, hipStream_t st);

struct FfnPlan;
mok_status launch_ffn_forward(const FfnPlan &p, void *workspace, const uint16_t *x, const uint8_t *x_elems,
                              const uint8_t *x_scales, const mok_weights &w, const uint16_t *addend, uint16_t *out,
                              uint16_t *h, hipStream_t st);
mok_status launch_ffn_backward(const FfnPlan &p, void *workspace, const uint16_t *x, const mok_weights &w,
                               const uint16_t *h, const uint16_t *dy, const uint16_t *addend, uint16_t *dx,
                               uint16_t *dw_gate, uint16_t *dw_up, uint16_t *dw_down, hipStream_t st);

}  // namespace mok
