// Forward of the gated feed-forward block for a few rows: see ffn_few.hip.
#pragma once
#include <hip/hip_runtime.h>

#include "ffn_plan.h"

namespace mok {

hipError_t ffn_few_forward(const FfnPlan &p, char *ws, const uint16_t *x, const mok_weights &w, const uint16_t *addend,
                           uint16_t *out, uint16_t *h, hipStream_t st);
hipError_t ffn_few_mx_forward(const FfnPlan &p, char *ws, const uint8_t *x_elems, const uint8_t *x_scales,
                              const mok_weights &w, const uint16_t *addend, uint16_t *out, uint16_t *h, hipStream_t st);

}  // namespace mok
