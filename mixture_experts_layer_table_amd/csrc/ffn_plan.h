// Host-side plan of the gated feed-forward block: sizes, the split of each
// product over its contraction axis, and the workspace layout (no HIP calls).
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/mok.h"

namespace mok {

// One product of T rows: tiles of bm x 256 outputs, the contraction axis cut
// into `splits` runs of `len` K-steps (32 values in BF16, 64 in MXFP8). With
// more than one run every tile writes fp32 partials that a second kernel adds
// in ascending order.
struct FfnSplit {
    int bm, splits, len;
};

// Workgroups of a product come in multiples of the dies (kXcds on the device side).
constexpr int kGridStep = 8;

// Most rows that take the few-rows kernels (ffn_few.hip).
constexpr int kFewRows = 2;

struct FfnPlan {
    int64_t T;
    int H, I;
    bool mx;
    FfnSplit gate_up, down, da, dx;
    int wgrad_bm;     // m-tile rows of the weight gradients
    bool grads_two;   // BF16, dx and the weight gradients on 128 rows: two workgroups a unit
    // few-rows forward: 0 runs where the tile kernels are taken instead;
    // BF16 gate/up: runs of few_run_rows rows of the weights
    int few_runs, few_run_rows;
    // workspace offsets (bytes); the forward and the backward overlay each other
    size_t part, a, dh, a_q, a_qs, dh_q, dh_qs, dy_q, dy_qs, total;
};

mok_status make_ffn_plan(int64_t T, int32_t H, int32_t I, int32_t precision, FfnPlan *p);

}  // namespace mok
