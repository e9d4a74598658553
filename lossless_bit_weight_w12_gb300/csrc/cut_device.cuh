// cut_device.cuh -- a token's weight after its row's cuts (RowCut), shared by the
// kernel that finds the cuts and the one that draws.
#pragma once

#include "draft_internal.h"
#include "sample_device.cuh"

namespace w12 {

// A whole number below 2^31 as an integer and in fp32 (it has 24 bits at most).
struct Weight {
    uint32_t whole;
    float f;
};

// The weight of token i with logit v (a NaN and -infinity have 0).
__device__ __forceinline__ Weight cut_weight(const RowCut &c, float v, int i) {
    const float y = expf(__fmul_rn(__fsub_rn(fminf(v, 3.402823466e38f), c.mx), c.inv_t)) * kOne31;
    // (the sum is rounded to a whole number; from 2^23 on y is one)
    const float f = y < 8388608.0f ? __fsub_rn(__fadd_rn(y, 8388608.0f), 8388608.0f) : y;
    const bool stays = (v > c.least || (v == c.least && i <= c.last)) && f >= c.floor;
    return Weight{stays ? __float2uint_rn(y) : 0u, stays ? f : 0.0f};
}

}  // namespace w12
