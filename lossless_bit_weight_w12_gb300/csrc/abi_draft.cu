// abi_draft.cu -- the extern "C" entry points of the calls around a draft
// model (include/w12.h: add and norm, 4-bit products, sampled verification):
// argument checks and dispatch.  Host code only.
#include <cuda_runtime.h>

#include "draft_internal.h"

namespace w12 {

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kLim31 = int64_t(1) << 31;

size_t size_of(int dtype) { return dtype == W12_F32 ? 4 : dtype == W12_BF16 ? 2 : 1; }

bool float_type(int dtype) { return dtype == W12_F32 || dtype == W12_BF16; }

}  // namespace

}  // namespace w12

using namespace w12;

extern "C" int w12_add_norm(const void *x, int64_t x_stride, int x_dtype, const void *delta, int64_t delta_stride,
                            int delta_dtype, const void *weight, int weight_dtype, float offset, float eps, int64_t rows,
                            int64_t dim, void *residual, int64_t residual_stride, void *out, int64_t out_stride,
                            int out_dtype, float *scale, void *stream) {
    if (!float_type(x_dtype) || (delta && !float_type(delta_dtype)) || (weight && !float_type(weight_dtype)) ||
        (out_dtype != W12_BF16 && out_dtype != W12_E4M3))
        return W12_ERR_ARG;
    if (!(eps >= 0.0f) || !(offset - offset == 0.0f) || !(eps - eps == 0.0f)) return W12_ERR_ARG;
    if (rows < 0 || rows >= kLim31 || dim < 1 || dim > W12_NORM_MAX_DIM) return W12_ERR_SHAPE;
    if (rows > 1 && (out_stride < dim || (residual && residual_stride < dim))) return W12_ERR_SHAPE;
    if (rows == 0) return W12_OK;
    if (!x || !out || (out_dtype == W12_E4M3) != (scale != nullptr)) return W12_ERR_ARG;
    if (!aligned(x, size_of(x_dtype)) || (delta && !aligned(delta, size_of(delta_dtype))) ||
        (weight && !aligned(weight, size_of(weight_dtype))) || (residual && !aligned(residual, size_of(x_dtype))) ||
        !aligned(out, size_of(out_dtype)) || !aligned(scale, 4))
        return W12_ERR_ALIGN;
    NormArgs a = {};
    a.x = x, a.delta = delta, a.weight = weight, a.residual = residual, a.out = out, a.scale = scale;
    a.x_stride = x_stride, a.delta_stride = delta_stride, a.residual_stride = residual_stride, a.out_stride = out_stride;
    a.rows = rows, a.dim = int32_t(dim), a.weight_f32 = weight && weight_dtype == W12_F32;
    a.eps = eps, a.offset = offset;
    // rows on 16-byte boundaries (e4m3: 8), whole eights of elements
    const auto rows_at = [&](const void *p, int64_t stride, size_t size, size_t to) {
        return !p || (aligned(p, to) && (rows == 1 || uint64_t(stride) * size % to == 0));
    };
    const bool vec = dim % 8 == 0 && rows_at(x, x_stride, size_of(x_dtype), 16) &&
                     rows_at(delta, delta_stride, size_of(delta_dtype), 16) && aligned(weight, 16) &&
                     rows_at(residual, residual_stride, size_of(x_dtype), 16) &&
                     rows_at(out, out_stride, size_of(out_dtype), out_dtype == W12_E4M3 ? 8 : 16);
    return launch_norm(a, x_dtype, delta ? delta_dtype : -1, out_dtype, vec, stream);
}
