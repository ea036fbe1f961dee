// Host-side plan of the products on blocks of 128: tiles and workspace (no HIP calls).
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/mok.h"

namespace mok {

struct BlkPlan {
    int64_t M;
    int N, K, E;
    bool f32;
    int bm;            // tile rows
    int few, few_w;    // tiles of 16 rows, and of 16 weight rows, of the few-rows kernel; 0: not taken
    int splits, run;   // runs of the contraction, joined by a second kernel; K-blocks of one (products by weights)
    size_t total;      // workspace bytes (0: none)
};

mok_status make_blk_matmul_plan(const mok_fp8_shape *s, BlkPlan *p);
mok_status make_blk_wgrad_plan(const mok_fp8_shape *s, BlkPlan *p);

}  // namespace mok
