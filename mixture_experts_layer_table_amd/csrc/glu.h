// The gated activation a = silu(g) * u and its gradient, one value.
#pragma once
#include "common.h"

namespace mok {

__device__ __forceinline__ float glu_forward(float g, float u) { return g * sigmoidf_(g) * u; }

struct GluGrad {
    float a, dg, du;
};
__device__ __forceinline__ GluGrad glu_backward(float da, float hg, float hu) {
    const float s = sigmoidf_(hg), sl = hg * s;
    return GluGrad{sl * hu, da * hu * s * (1.0f + hg * (1.0f - s)), da * sl};
}

}  // namespace mok
