// draft_internal.h -- declarations shared by the calls around a draft model
// (add and norm, 4-bit products, sampled verification): argument blocks of
// the kernels and their launchers.  Not installed.
#pragma once

#include <cstddef>
#include <cstdint>

#include "step_internal.h"

namespace w12 {

struct NormArgs {
    const void *x, *delta, *weight;
    void *residual, *out;
    float *scale;
    int64_t x_stride, delta_stride, residual_stride, out_stride;  // elements per row
    int64_t rows;
    int32_t dim;
    int32_t weight_f32;
    float eps, offset;
};
// delta_dtype -1: no delta.  vec: every row of every tensor starts on a
// 16-byte boundary and dim is a multiple of 8.
int launch_norm(const NormArgs &a, int x_dtype, int delta_dtype, int out_dtype, bool vec, void *stream);

}  // namespace w12
