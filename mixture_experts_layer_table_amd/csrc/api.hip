// C ABI entry points: argument validation on the host, then launches.
#include <algorithm>
#include <cstdint>

#include "ffn_plan.h"
#include "kernels.h"
#include "plan.h"

using namespace mok;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool dev_ok(const void *p) { return p != nullptr && aligned16(p); }
bool dev_ok_or_null(const void *p) { return aligned16(p); }

bool stream_ok(int32_t dtype) { return dtype == MOK_STREAM_BF16 || dtype == MOK_STREAM_F32; }
// p in [0, 1); the state is read only where something can be dropped
bool drop_ok(float p, const uint64_t *rng) {
    return p >= 0.0f && p < 1.0f && (p == 0.0f || (rng && (reinterpret_cast<uintptr_t>(rng) & 7u) == 0));
}

// Bytes [p, p + n) of a buffer (null: none), to refuse outputs that overlap what other threads still read.
struct Span {
    const void *p;
    size_t n;
};
// The dropout state, where it is read.
Span rng_span(float p, const uint64_t *rng) { return {p > 0.0f ? rng : nullptr, 16}; }
bool overlap(Span a, Span b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}
// The two may be one and the same buffer, but not partly overlap.
bool overlap_partly(Span a, Span b) { return overlap(a, b) && !(a.p == b.p && a.n == b.n); }
template <size_t N>
bool any_overlap(Span a, const Span (&others)[N]) {
    for (const Span &o : others)
        if (overlap(a, o)) return true;
    return false;
}
// No two of the outputs overlap.
template <size_t N>
bool apart(const Span (&outs)[N]) {
    for (size_t i = 0; i < N; ++i)
        for (size_t j = i + 1; j < N; ++j)
            if (overlap(outs[i], outs[j])) return false;
    return true;
}

}  // namespace

extern "C" {

mok_status mok_config_default(mok_config *cfg) {
    if (!cfg) return MOK_ERROR_INVALID_VALUE;
    cfg->minibatch_rows = 512;
    cfg->precision = MOK_BF16;
    cfg->macrobatch_tokens = 0;
    cfg->ring_bytes = int64_t(256) << 20;
    cfg->capacity_multiplier = 1.0f;
    cfg->debug_flags = 0;
    cfg->persistent_workgroups = 0;
    return MOK_OK;
}

mok_status mok_config_autosize(mok_config *cfg, const mok_shape *shape, int32_t n_cu) {
    if (!cfg || !shape) return MOK_ERROR_INVALID_VALUE;
    const int64_t units = n_cu > 0 ? n_cu : 256;
    // Validate the shape and the other knobs with the smallest mini-batch and
    // an unbounded ring; the plan also gives the tile rows and the row bytes.
    mok_config probe = *cfg;
    probe.minibatch_rows = 16;
    probe.ring_bytes = int64_t(1) << 50;
    Plan p;
    mok_status s = make_plan(&probe, shape, &p);
    if (s != MOK_OK) return s;
    const int64_t BM = p.tile.BM;
    const int64_t rows = (2 * units * BM * kTileN + 2 * (int64_t)p.I - 1) / (2 * (int64_t)p.I);
    int64_t mb = (rows + BM - 1) / BM * BM;
    const int64_t macro_rows = ((int64_t)p.k * p.MT + 15) / 16 * 16;
    mb = std::max<int64_t>(16, std::min(mb, macro_rows));
    if (mb > (int64_t(1) << 30)) return MOK_ERROR_INVALID_VALUE;
    mok_config out = *cfg;
    out.minibatch_rows = (int32_t)mb;
    const int64_t two_slots = 2 * mb * (int64_t)p.ring_row_bytes;
    if (out.ring_bytes < two_slots) out.ring_bytes = two_slots;
    s = make_plan(&out, shape, &p);
    if (s != MOK_OK) return s;
    *cfg = out;
    return MOK_OK;
}

mok_status mok_query_sizes(const mok_config *cfg, const mok_shape *shape, size_t *workspace_bytes,
                           size_t *schedule_bytes, size_t *fwd_ctx_bytes) {
    Plan p;
    const mok_status s = make_plan(cfg, shape, &p);
    if (s != MOK_OK) return s;
    if (workspace_bytes) *workspace_bytes = p.w_total;
    if (schedule_bytes) *schedule_bytes = p.s_total;
    if (fwd_ctx_bytes) *fwd_ctx_bytes = p.c_total;
    return MOK_OK;
}

mok_status mok_schedule_layout_query(const mok_config *cfg, const mok_shape *shape, mok_schedule_layout *l) {
    if (!l) return MOK_ERROR_INVALID_VALUE;
    Plan p;
    const mok_status s = make_plan(cfg, shape, &p);
    if (s != MOK_OK) return s;
    l->R = p.R;
    l->NM = p.NM;
    l->G = p.G;
    l->cap = p.cap;
    l->status = p.s_status;
    l->n_seg = p.s_nseg;
    l->counts = p.s_counts;
    l->offsets = p.s_offsets;
    l->mcounts = p.s_mcounts;
    l->moffsets = p.s_moffsets;
    l->perm = p.s_perm;
    l->inv = p.s_inv;
    l->canon = p.s_canon;
    l->mb_start = p.s_mbstart;
    l->segments = p.s_segments;
    l->total_bytes = p.s_total;
    return MOK_OK;
}

mok_status mok_build_schedule(const mok_config *cfg, const mok_shape *shape, const int32_t *topk_ids,
                              void *schedule, size_t schedule_bytes, void *stream) {
    Plan p;
    mok_status s = make_plan(cfg, shape, &p);
    if (s != MOK_OK) return s;
    if (!dev_ok(schedule) || (p.R > 0 && !dev_ok(topk_ids))) return MOK_ERROR_INVALID_VALUE;
    if (schedule_bytes < p.s_total) return MOK_ERROR_BUFFER_TOO_SMALL;
    (void)hipGetLastError();   // drop an earlier, unrelated error of this thread
    return launch_build_schedule(p, topk_ids, schedule, static_cast<hipStream_t>(stream));
}

static mok_status check_weights(const Plan &p, const mok_weights *w) {
    if (!w) return MOK_ERROR_INVALID_VALUE;
    if (p.precision == MOK_BF16) {
        if (!dev_ok(w->w_gate) || !dev_ok(w->w_up) || !dev_ok(w->w_down)) return MOK_ERROR_INVALID_VALUE;
    } else {
        if (!dev_ok(w->gate_elems) || !dev_ok(w->gate_scales) || !dev_ok(w->up_elems) || !dev_ok(w->up_scales) ||
            !dev_ok(w->down_elems) || !dev_ok(w->down_scales))
            return MOK_ERROR_INVALID_VALUE;
    }
    return MOK_OK;
}

mok_status mok_forward(const mok_config *cfg, const mok_shape *shape, const void *schedule, size_t schedule_bytes,
                       void *workspace, size_t workspace_bytes, const void *x, const float *topk_w,
                       const mok_weights *w, void *out, void *fwd_ctx, size_t fwd_ctx_bytes, void *stream) {
    Plan p;
    mok_status s = make_plan(cfg, shape, &p);
    if (s != MOK_OK) return s;
    if ((s = check_weights(p, w)) != MOK_OK && !(p.debug & MOK_DEBUG_IDENTITY_EXPERT)) return s;
    if (!dev_ok(schedule) || !dev_ok(workspace) || !dev_ok(fwd_ctx)) return MOK_ERROR_INVALID_VALUE;
    if (p.R > 0 && (!dev_ok(x) || !dev_ok(topk_w) || !dev_ok(out))) return MOK_ERROR_INVALID_VALUE;
    if (schedule_bytes < p.s_total || workspace_bytes < p.w_total || fwd_ctx_bytes < p.c_total)
        return MOK_ERROR_BUFFER_TOO_SMALL;
    (void)hipGetLastError();
    if ((s = launch_schedule_check(p, schedule, static_cast<hipStream_t>(stream))) != MOK_OK) return s;
    return launch_forward(p, schedule, workspace, static_cast<const uint16_t *>(x), topk_w, *w,
                          static_cast<uint16_t *>(out), fwd_ctx, static_cast<hipStream_t>(stream));
}

mok_status mok_backward(const mok_config *cfg, const mok_shape *shape, const void *schedule, size_t schedule_bytes,
                        void *workspace, size_t workspace_bytes, const void *x, const float *topk_w,
                        const mok_weights *w,
                        const void *fwd_ctx, size_t fwd_ctx_bytes, const void *dy, void *dx, void *dw_gate,
                        void *dw_up, void *dw_down, float *dtopk_w, void *stream) {
    Plan p;
    mok_status s = make_plan(cfg, shape, &p);
    if (s != MOK_OK) return s;
    if (p.debug & MOK_DEBUG_IDENTITY_EXPERT) return MOK_ERROR_UNSUPPORTED;
    if ((s = check_weights(p, w)) != MOK_OK) return s;
    if (!dev_ok(schedule) || !dev_ok(workspace) || !dev_ok(fwd_ctx)) return MOK_ERROR_INVALID_VALUE;
    if (!dev_ok(dw_gate) || !dev_ok(dw_up) || !dev_ok(dw_down)) return MOK_ERROR_INVALID_VALUE;
    if (p.R > 0 && (!dev_ok(x) || !dev_ok(topk_w) || !dev_ok(dy) || !dev_ok(dx) || !dev_ok(dtopk_w)))
        return MOK_ERROR_INVALID_VALUE;
    if (schedule_bytes < p.s_total || workspace_bytes < p.w_total || fwd_ctx_bytes < p.c_total)
        return MOK_ERROR_BUFFER_TOO_SMALL;
    (void)hipGetLastError();
    if ((s = launch_schedule_check(p, schedule, static_cast<hipStream_t>(stream))) != MOK_OK) return s;
    return launch_backward(p, schedule, workspace, static_cast<const uint16_t *>(x), topk_w, *w, fwd_ctx,
                           static_cast<const uint16_t *>(dy), static_cast<uint16_t *>(dx),
                           static_cast<uint16_t *>(dw_gate), static_cast<uint16_t *>(dw_up),
                           static_cast<uint16_t *>(dw_down), dtopk_w, static_cast<hipStream_t>(stream));
}

mok_status mok_mxfp8_quantize(const void *src, int64_t batch, int64_t rows, int64_t K, int32_t src_is_k_by_rows,
                              uint8_t *elems, uint8_t *scales, void *stream) {
    if (batch < 0 || rows < 0 || K < 0 || K % 32) return MOK_ERROR_INVALID_VALUE;
    if (src_is_k_by_rows != 0 && src_is_k_by_rows != 1) return MOK_ERROR_INVALID_VALUE;
    if (batch * rows * K == 0) return MOK_OK;
    if (!dev_ok(src) || !dev_ok(elems) || !scales) return MOK_ERROR_INVALID_VALUE;
    (void)hipGetLastError();
    return launch_mxfp8_quantize(static_cast<const uint16_t *>(src), batch, rows, K, src_is_k_by_rows == 1, elems,
                                 scales, static_cast<hipStream_t>(stream));
}

mok_status mok_route(const float *logits, int64_t T, int32_t E, int32_t k, int32_t *topk_ids, float *topk_w,
                     void *stream) {
    if (T < 0 || E < 1 || E > 1024 || k < 1 || k > E || k > 64) return MOK_ERROR_INVALID_VALUE;
    if (T == 0) return MOK_OK;
    if (!aligned4(logits) || !aligned4(topk_ids) || !aligned4(topk_w)) return MOK_ERROR_INVALID_VALUE;
    (void)hipGetLastError();
    return launch_route(logits, T, E, k, topk_ids, topk_w, static_cast<hipStream_t>(stream));
}

mok_status mok_route_backward(const int32_t *topk_ids, const float *topk_w, const float *dtopk_w, int64_t T,
                              int32_t E, int32_t k, float *dlogits, void *stream) {
    if (T < 0 || E < 1 || E > 1024 || k < 1 || k > E || k > 64) return MOK_ERROR_INVALID_VALUE;
    if (T == 0) return MOK_OK;
    if (!aligned4(topk_ids) || !aligned4(topk_w) || !aligned4(dtopk_w) || !aligned4(dlogits))
        return MOK_ERROR_INVALID_VALUE;
    (void)hipGetLastError();
    return launch_route_backward(topk_ids, topk_w, dtopk_w, T, E, k, dlogits, static_cast<hipStream_t>(stream));
}

mok_status mok_dropout(const void *x, const void *residual, int64_t n, float p, const uint64_t *rng,
                       int32_t stream_dtype, void *out, void *stream) {
    if (n < 0 || n > kMaxDropout || !stream_ok(stream_dtype) || !drop_ok(p, rng)) return MOK_ERROR_INVALID_VALUE;
    if (n == 0) return MOK_OK;
    if (!dev_ok(x) || !dev_ok_or_null(residual) || !dev_ok(out)) return MOK_ERROR_INVALID_VALUE;
    const bool f32 = stream_dtype == MOK_STREAM_F32;
    const size_t sb = (size_t)n * (f32 ? 4 : 2);
    if (overlap_partly({out, sb}, {residual, sb}) || overlap_partly({out, sb}, {x, (size_t)n * 2}) ||
        overlap({out, sb}, rng_span(p, rng)))
        return MOK_ERROR_INVALID_VALUE;
    (void)hipGetLastError();
    return launch_dropout(static_cast<const uint16_t *>(x), residual, n, p, rng, f32, out,
                          static_cast<hipStream_t>(stream));
}

mok_status mok_dropout_backward(const void *dy, int64_t n, float p, const uint64_t *rng, int32_t stream_dtype,
                                void *dx, void *stream) {
    if (n < 0 || n > kMaxDropout || !stream_ok(stream_dtype) || !drop_ok(p, rng)) return MOK_ERROR_INVALID_VALUE;
    if (n == 0) return MOK_OK;
    if (!dev_ok(dy) || !dev_ok(dx)) return MOK_ERROR_INVALID_VALUE;
    const bool f32 = stream_dtype == MOK_STREAM_F32;
    const Span sdx{dx, (size_t)n * 2};
    if (overlap_partly(sdx, {dy, (size_t)n * (f32 ? 4 : 2)}) || overlap(sdx, rng_span(p, rng)))
        return MOK_ERROR_INVALID_VALUE;
    (void)hipGetLastError();
    return launch_dropout_backward(dy, n, p, rng, f32, static_cast<uint16_t *>(dx), static_cast<hipStream_t>(stream));
}

static bool norm_shape_ok(const mok_norm_shape *s) {
    return s && s->T >= 0 && s->T < (int64_t(1) << 31) && s->H > 0 && s->H <= kNormMaxH && s->H % 8 == 0 &&
           stream_ok(s->stream_dtype) && s->eps >= 0.0f && s->eps <= 3.4e38f && s->p >= 0.0f && s->p < 1.0f;
}

mok_status mok_add_rmsnorm(const mok_norm_shape *shape, const void *x, const void *residual, const void *weight,
                           const uint64_t *rng, void *sum, void *y, uint8_t *y_elems, uint8_t *y_scales, float *rstd,
                           void *stream) {
    if (!norm_shape_ok(shape) || !drop_ok(shape->p, rng)) return MOK_ERROR_INVALID_VALUE;
    if (shape->T == 0) return MOK_OK;   // empty buffers may be NULL
    if ((y_elems == nullptr) != (y_scales == nullptr) || (!y && !y_elems)) return MOK_ERROR_INVALID_VALUE;
    if (y_elems && shape->H % 32) return MOK_ERROR_INVALID_VALUE;
    if (!dev_ok(x) || !dev_ok_or_null(residual) || !dev_ok(weight) || !dev_ok_or_null(sum) || !dev_ok_or_null(y) ||
        !dev_ok_or_null(y_elems) || !dev_ok_or_null(y_scales) || !aligned4(rstd))
        return MOK_ERROR_INVALID_VALUE;
    const size_t n = (size_t)shape->T * shape->H, h2 = (size_t)shape->H * 2;
    const bool f32 = shape->stream_dtype == MOK_STREAM_F32;
    const Span sx{x, n * 2}, sr{residual, n * (f32 ? 4 : 2)}, ss{sum, n * (f32 ? 4 : 2)};
    const Span rest[] = {{y, n * 2}, {y_elems, n}, {y_scales, n / 32}, {rstd, (size_t)shape->T * 4}};
    const Span outs[] = {ss, rest[0], rest[1], rest[2], rest[3]};
    const Span ins[] = {sx, sr, {weight, h2}, rng_span(shape->p, rng)};
    if (!apart(outs) || overlap_partly(ss, sx) || overlap_partly(ss, sr) || overlap(ss, ins[2]) || overlap(ss, ins[3]))
        return MOK_ERROR_INVALID_VALUE;
    for (const Span &o : rest)
        if (any_overlap(o, ins)) return MOK_ERROR_INVALID_VALUE;
    (void)hipGetLastError();
    NormCall c{};
    c.T = shape->T;
    c.H = shape->H;
    c.eps = shape->eps;
    c.p = shape->p;
    c.f32_stream = f32;
    c.x = static_cast<const uint16_t *>(x);
    c.residual = residual;
    c.weight = static_cast<const uint16_t *>(weight);
    c.rng = rng;
    c.sum = sum;
    c.y = static_cast<uint16_t *>(y);
    c.elems = y_elems;
    c.scales = y_scales;
    c.rstd = rstd;
    return launch_add_rmsnorm(c, static_cast<hipStream_t>(stream));
}

mok_status mok_add_rmsnorm_backward_size(const mok_norm_shape *shape, size_t *workspace_bytes) {
    if (!norm_shape_ok(shape) || !workspace_bytes) return MOK_ERROR_INVALID_VALUE;
    *workspace_bytes = std::max<size_t>(256, (size_t)norm_backward_shares(shape->T, shape->H) * shape->H * 4);
    return MOK_OK;
}

mok_status mok_add_rmsnorm_backward(const mok_norm_shape *shape, void *workspace, size_t workspace_bytes,
                                    const void *dy, const void *sum, const void *weight, const float *rstd,
                                    const void *dsum, const uint64_t *rng, void *dresidual, void *dx, float *dweight,
                                    void *stream) {
    size_t need = 0;
    const mok_status s = mok_add_rmsnorm_backward_size(shape, &need);
    if (s != MOK_OK) return s;
    if (!drop_ok(shape->p, rng) || !dev_ok(workspace) || !dev_ok(dweight)) return MOK_ERROR_INVALID_VALUE;
    if (shape->T > 0 && (!dev_ok(dy) || !dev_ok(sum) || !dev_ok(weight) || !aligned4(rstd) || !dev_ok_or_null(dsum) ||
                         !dev_ok_or_null(dresidual) || !dev_ok_or_null(dx)))
        return MOK_ERROR_INVALID_VALUE;
    if (workspace_bytes < need) return MOK_ERROR_BUFFER_TOO_SMALL;
    const size_t n = (size_t)shape->T * shape->H, h2 = (size_t)shape->H * 2;
    const bool f32 = shape->stream_dtype == MOK_STREAM_F32;
    const size_t sb = n * (f32 ? 4 : 2);
    const Span sres{dresidual, sb}, sdx{dx, n * 2}, sdw{dweight, 2 * h2}, sws{workspace, need};
    const Span sdy{dy, n * 2}, sds{dsum, sb}, sin{sum, sb}, sw{weight, h2}, sr{rstd, (size_t)shape->T * 4};
    const Span sg = rng_span(shape->p, rng);
    const Span outs[] = {sres, sdx, sdw, sws}, ins[] = {sdy, sds, sin, sw, sr, sg}, fixed[] = {sin, sw, sr, sg};
    if (!apart(outs) || any_overlap(sres, fixed) || any_overlap(sdx, fixed) || any_overlap(sdw, ins) ||
        any_overlap(sws, ins) || overlap(sres, sdy) || overlap_partly(sres, sds) || overlap(sdx, sds) ||
        overlap_partly(sdx, sdy))
        return MOK_ERROR_INVALID_VALUE;
    (void)hipGetLastError();
    NormBackwardCall c{};
    c.T = shape->T;
    c.H = shape->H;
    c.p = shape->p;
    c.f32_stream = f32;
    c.dy = static_cast<const uint16_t *>(dy);
    c.sum = sum;
    c.dsum = dsum;
    c.weight = static_cast<const uint16_t *>(weight);
    c.rstd = rstd;
    c.rng = rng;
    c.dres = dresidual;
    c.dx = static_cast<uint16_t *>(dx);
    c.dweight = dweight;
    c.part = static_cast<float *>(workspace);
    return launch_add_rmsnorm_backward(c, static_cast<hipStream_t>(stream));
}

static mok_status ffn_plan_of(const mok_ffn_shape *shape, FfnPlan *p) {
    return shape ? make_ffn_plan(shape->T, shape->H, shape->I, shape->precision, p) : MOK_ERROR_INVALID_VALUE;
}

static bool ffn_weights_ok(const FfnPlan &p, const mok_weights *w) {
    if (!w) return false;
    if (!p.mx) return dev_ok(w->w_gate) && dev_ok(w->w_up) && dev_ok(w->w_down);
    return dev_ok(w->gate_elems) && dev_ok(w->gate_scales) && dev_ok(w->up_elems) && dev_ok(w->up_scales) &&
           dev_ok(w->down_elems) && dev_ok(w->down_scales);
}

// The weights' buffers, in either precision (unused pointers are skipped).
struct FfnWeightSpans {
    Span s[6];
};
static FfnWeightSpans ffn_weight_spans(const FfnPlan &p, const mok_weights *w) {
    const size_t n = (size_t)p.H * p.I;
    if (!p.mx) return {{{w->w_gate, n * 2}, {w->w_up, n * 2}, {w->w_down, n * 2}, {}, {}, {}}};
    return {{{w->gate_elems, n}, {w->gate_scales, n / 32}, {w->up_elems, n}, {w->up_scales, n / 32},
             {w->down_elems, n}, {w->down_scales, n / 32}}};
}

mok_status mok_ffn_query_size(const mok_ffn_shape *shape, size_t *workspace_bytes) {
    FfnPlan p;
    const mok_status s = ffn_plan_of(shape, &p);
    if (s != MOK_OK) return s;
    if (!workspace_bytes) return MOK_ERROR_INVALID_VALUE;
    *workspace_bytes = p.total;
    return MOK_OK;
}

mok_status mok_ffn_forward(const mok_ffn_shape *shape, void *workspace, size_t workspace_bytes, const void *x,
                           const uint8_t *x_elems, const uint8_t *x_scales, const mok_weights *w, const void *addend,
                           void *out, void *h, void *stream) {
    FfnPlan p;
    const mok_status s = ffn_plan_of(shape, &p);
    if (s != MOK_OK) return s;
    if (!ffn_weights_ok(p, w) || !dev_ok(workspace)) return MOK_ERROR_INVALID_VALUE;
    if (p.T > 0) {
        if (p.mx ? (!dev_ok(x_elems) || !dev_ok(x_scales)) : !dev_ok(x)) return MOK_ERROR_INVALID_VALUE;
        if (!dev_ok_or_null(addend) || !dev_ok(out) || !dev_ok_or_null(h)) return MOK_ERROR_INVALID_VALUE;
    }
    if (workspace_bytes < p.total) return MOK_ERROR_BUFFER_TOO_SMALL;
    if (p.T == 0) return MOK_OK;
    const size_t n = (size_t)p.T * p.H;
    const Span so{out, n * 2}, sh{h, (size_t)p.T * p.I * 4}, sws{workspace, p.total}, sadd{addend, n * 2};
    const Span outs[] = {so, sh, sws};
    const Span ins[] = {
        {p.mx ? nullptr : x, n * 2}, {p.mx ? x_elems : nullptr, n}, {p.mx ? x_scales : nullptr, n / 32}};
    const FfnWeightSpans ws = ffn_weight_spans(p, w);
    if (!apart(outs) || overlap_partly(so, sadd) || overlap(sh, sadd) || overlap(sws, sadd))
        return MOK_ERROR_INVALID_VALUE;
    for (const Span &o : outs)
        if (any_overlap(o, ins) || any_overlap(o, ws.s)) return MOK_ERROR_INVALID_VALUE;
    (void)hipGetLastError();
    return launch_ffn_forward(p, workspace, static_cast<const uint16_t *>(x), x_elems, x_scales, *w,
                              static_cast<const uint16_t *>(addend), static_cast<uint16_t *>(out),
                              static_cast<uint16_t *>(h), static_cast<hipStream_t>(stream));
}

mok_status mok_ffn_backward(const mok_ffn_shape *shape, void *workspace, size_t workspace_bytes, const void *x,
                            const mok_weights *w, const void *h, const void *dy, const void *addend, void *dx,
                            void *dw_gate, void *dw_up, void *dw_down, void *stream) {
    FfnPlan p;
    const mok_status s = ffn_plan_of(shape, &p);
    if (s != MOK_OK) return s;
    if (!ffn_weights_ok(p, w) || !dev_ok(workspace)) return MOK_ERROR_INVALID_VALUE;
    if (!dev_ok(dw_gate) || !dev_ok(dw_up) || !dev_ok(dw_down)) return MOK_ERROR_INVALID_VALUE;
    if (p.T > 0 && (!dev_ok(x) || !dev_ok(h) || !dev_ok(dy) || !dev_ok_or_null(addend) || !dev_ok(dx)))
        return MOK_ERROR_INVALID_VALUE;
    if (workspace_bytes < p.total) return MOK_ERROR_BUFFER_TOO_SMALL;
    const size_t n = (size_t)p.T * p.H, wb = (size_t)p.H * p.I * 2;
    const Span sdx{dx, n * 2}, sws{workspace, p.total}, sadd{addend, n * 2};
    const Span outs[] = {sdx, {dw_gate, wb}, {dw_up, wb}, {dw_down, wb}, sws};
    const Span ins[] = {{x, n * 2}, {h, (size_t)p.T * p.I * 4}, {dy, n * 2}};
    const FfnWeightSpans ws = ffn_weight_spans(p, w);
    if (!apart(outs) || overlap_partly(sdx, sadd)) return MOK_ERROR_INVALID_VALUE;
    for (const Span &o : outs)
        if (any_overlap(o, ins) || any_overlap(o, ws.s) || (o.p != dx && overlap(o, sadd)))
            return MOK_ERROR_INVALID_VALUE;
    (void)hipGetLastError();
    return launch_ffn_backward(p, workspace, static_cast<const uint16_t *>(x), *w, static_cast<const uint16_t *>(h),
                               static_cast<const uint16_t *>(dy), static_cast<const uint16_t *>(addend),
                               static_cast<uint16_t *>(dx), static_cast<uint16_t *>(dw_gate),
                               static_cast<uint16_t *>(dw_up), static_cast<uint16_t *>(dw_down),
                               static_cast<hipStream_t>(stream));
}

const char *mok_status_string(mok_status status) {
    switch (status) {
        case MOK_OK: return "MOK_OK";
        case MOK_ERROR_INVALID_VALUE: return "MOK_ERROR_INVALID_VALUE";
        case MOK_ERROR_UNSUPPORTED: return "MOK_ERROR_UNSUPPORTED";
        case MOK_ERROR_BUFFER_TOO_SMALL: return "MOK_ERROR_BUFFER_TOO_SMALL";
        case MOK_ERROR_LAUNCH_FAILED: return "MOK_ERROR_LAUNCH_FAILED";
    }
    return "MOK_ERROR_UNKNOWN";
}

}  // extern "C"
