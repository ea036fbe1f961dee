// Plan of the products on blocks of 128: see fp8_plan.h.
#include "fp8_plan.h"

#include <algorithm>

namespace mok {

namespace {

bool widths_ok(const mok_fp8_shape *s) {
    return s && s->M >= 0 && s->N > 0 && s->K > 0 && s->N % 16 == 0 && s->K % 16 == 0 && s->N <= (1 << 20) &&
           s->K <= (1 << 20) && s->E >= 0 && s->E <= 4096 &&
           (s->out_dtype == MOK_STREAM_BF16 || s->out_dtype == MOK_STREAM_F32);
}

void fill(const mok_fp8_shape *s, BlkPlan *p) {
    *p = BlkPlan{};
    p->M = s->M;
    p->N = s->N;
    p->K = s->K;
    p->E = s->E;
    p->f32 = s->out_dtype == MOK_STREAM_F32;
    p->bm = 256;
    p->total = 256;
}

// Workgroups stay within one grid of fewer than 2^32 threads.
constexpr int64_t kMostTiles = (1 << 23) - 64;
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

mok_status make_blk_matmul_plan(const mok_fp8_shape *s, BlkPlan *p) {
    if (!widths_ok(s) || s->M >= (int64_t(1) << 31)) return MOK_ERROR_INVALID_VALUE;
    fill(s, p);
    const int64_t per = s->M / std::max(s->E, 1);   // rows of an expert in the mean
    if (per <= 128 || p->f32) p->bm = 128;
    if ((ceil_div(s->M, p->bm) + s->E) * ceil_div(s->N, 256) > kMostTiles) return MOK_ERROR_UNSUPPORTED;
    return MOK_OK;
}

mok_status make_blk_wgrad_plan(const mok_fp8_shape *s, BlkPlan *p) {
    if (!widths_ok(s) || s->M >= (int64_t(1) << 23) || s->M % 16) return MOK_ERROR_INVALID_VALUE;
    fill(s, p);
    if (s->N <= 128 || p->f32) p->bm = 128;
    if ((ceil_div(s->N, p->bm) * ceil_div(s->K, 256) + 8) * std::max(s->E, 1) > kMostTiles)
        return MOK_ERROR_UNSUPPORTED;
    return MOK_OK;
}

}  // namespace mok
