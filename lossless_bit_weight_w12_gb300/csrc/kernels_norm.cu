// kernels_norm.cu -- residual addition and root-mean-square norm of rows, out
// in bf16 or in e4m3 with one fp32 scale per row.
//
//   h = x + delta,  r = 1 / sqrt(mean(h^2) + eps),  y = (h (weight + offset)) r
//
// One CTA per row, the row in registers: every tensor is read or written once.
// The e4m3 scale needs the largest |y|; as r is one positive number for the
// row and a rounded product does not decrease with its factor, it is the
// rounded product of r and the largest |h (weight + offset)|, so one block
// reduction carries both the sum of squares and that maximum (as the bits of
// |.|, which order like the numbers and put NaN above infinity).
//
// The sum of squares is fp32.  Where it overflows, the row is scaled by 2^-80
// in its registers and reduced once more (eps is below every rounding there).
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "draft_internal.h"
#include "step_device.cuh"

namespace w12 {

namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyRow = 1e-30f;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint4 load16(const void *p) {  // (x may be written by this CTA: not the read-only path)
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

// Elements i .. i + 7 of a row.
template <bool F32>
__device__ __forceinline__ void load8(const void *row, int i, float (&v)[8]) {
    if (F32) {
        const uint4 a = load16(static_cast<const float *>(row) + i), b = load16(static_cast<const float *>(row) + i + 4);
        v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
    } else {
        const uint4 a = load16(static_cast<const uint16_t *>(row) + i);
        v[0] = bf_lo(a.x), v[1] = bf_hi(a.x), v[2] = bf_lo(a.y), v[3] = bf_hi(a.y);
        v[4] = bf_lo(a.z), v[5] = bf_hi(a.z), v[6] = bf_lo(a.w), v[7] = bf_hi(a.w);
    }
}

template <bool F32>
__device__ __forceinline__ float load1(const void *row, int i) {
    return F32 ? static_cast<const float *>(row)[i] : bf16_bits_to_float(static_cast<const uint16_t *>(row)[i]);
}

template <bool F32>
__device__ __forceinline__ void store1(void *row, int i, float v) {
    if (F32)
        static_cast<float *>(row)[i] = v;
    else
        static_cast<uint16_t *>(row)[i] = uint16_t(pack_bf16(v, 0.0f));
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {  // the first in the low byte
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// The row's sum of squares and largest |h (weight + offset)| (as bits).
__device__ __forceinline__ void reduce(float &sum, uint32_t &top, float *s_sum, uint32_t *s_top) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) s_sum[warp] = sum, s_top[warp] = top;
    __syncthreads();
    sum = lane < warps ? s_sum[lane] : 0.0f;
    top = lane < warps ? s_top[lane] : 0u;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
}

// E: elements of a row per thread.  VEC: eight consecutive ones at a time
// (chunk tid + q blockDim), else one (element tid + q blockDim).  XF, DF: x
// and delta in fp32 (DF -1: no delta).
template <int E, bool VEC, bool XF, int DF, bool E4M3>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float s_sum[2][32];
    __shared__ uint32_t s_top[2][32];
    const int tid = threadIdx.x, step = blockDim.x;
    const int64_t r = blockIdx.x;
    constexpr int W = VEC ? 8 : 1, Q = E / W;
    pdl_launch_dependents();
    pdl_wait_previous();
    const auto at = [](const void *p, int64_t elements, bool f32) {
        return static_cast<const unsigned char *>(p) + elements * (f32 ? 4 : 2);
    };
    const void *x = at(a.x, r * a.x_stride, XF);
    const void *d = DF >= 0 ? at(a.delta, r * a.delta_stride, DF > 0) : nullptr;
    float h[Q][W], w[Q][W];
    int i[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        i[q] = (tid + q * step) * W;
        if (i[q] < a.dim) {
            if constexpr (VEC) {
                load8<XF>(x, i[q], h[q]);
            } else {
                h[q][0] = load1<XF>(x, i[q]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) h[q][j] = 0.0f;
        }
    }
    if constexpr (DF >= 0) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (i[q] < a.dim) {
                float y[W];
                if constexpr (VEC) {
                    load8<(DF > 0)>(d, i[q], y);
                } else {
                    y[0] = load1<(DF > 0)>(d, i[q]);
                }
#pragma unroll
                for (int j = 0; j < W; ++j) h[q][j] += y[j];
            }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[q][j] = 1.0f;
        if (a.weight && i[q] < a.dim) {
            if constexpr (VEC) {
                if (a.weight_f32)
                    load8<true>(a.weight, i[q], w[q]);
                else
                    load8<false>(a.weight, i[q], w[q]);
            } else {
                w[q][0] = a.weight_f32 ? load1<true>(a.weight, i[q]) : load1<false>(a.weight, i[q]);
            }
        }
#pragma unroll
        for (int j = 0; j < W; ++j) w[q][j] += a.offset;
    }
    if (a.residual) {
        void *o = static_cast<unsigned char *>(a.residual) + r * a.residual_stride * (XF ? 4 : 2);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (i[q] < a.dim) {
                if constexpr (VEC && XF) {
                    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(o) + i[q]);
                    p[0] = make_float4(h[q][0], h[q][1], h[q][2], h[q][3]);
                    p[1] = make_float4(h[q][4], h[q][5], h[q][6], h[q][7]);
                } else if constexpr (VEC) {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(o) + i[q]) =
                        make_uint4(pack_bf16(h[q][0], h[q][1]), pack_bf16(h[q][2], h[q][3]), pack_bf16(h[q][4], h[q][5]),
                                   pack_bf16(h[q][6], h[q][7]));
                } else {
                    store1<XF>(o, i[q], h[q][0]);
                }
            }
    }
    float sum, eps = a.eps;
    uint32_t top;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        sum = 0.0f, top = 0u;
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int j = 0; j < W; ++j) {
                sum = fmaf(h[q][j], h[q][j], sum);
                if (E4M3) top = max(top, __float_as_uint(h[q][j] * w[q][j]) & 0x7FFFFFFFu);
            }
        reduce(sum, top, s_sum[pass], s_top[pass]);
        if (pass == 1 || sum != INFINITY) break;
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int j = 0; j < W; ++j) h[q][j] *= 0x1p-80f;
        eps = 0.0f;
    }
    const float rs = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(sum, float(a.dim)) + eps));
    if constexpr (E4M3) {
        const float amax = __uint_as_float(top) * rs;
        const bool bad = !(amax <= 3.402823466e38f), some = amax > kTinyRow;
        const float inv = !bad && some ? __fdiv_rn(kE4m3Max, amax) : 0.0f;
        if (tid == 0) a.scale[r] = bad ? __uint_as_float(0x7FC00000u) : some ? __fdiv_rn(amax, kE4m3Max) : 0.0f;
        uint8_t *o = static_cast<uint8_t *>(a.out) + r * a.out_stride;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (i[q] < a.dim) {
                float y[W];
                // (inv 0: zeros, also where the row holds a NaN or an infinity)
#pragma unroll
                for (int j = 0; j < W; ++j) y[j] = inv > 0.0f ? h[q][j] * w[q][j] * rs * inv : 0.0f;
                if constexpr (VEC) {
                    *reinterpret_cast<uint2 *>(o + i[q]) = make_uint2(pack_e4m3(y[0], y[1]) | pack_e4m3(y[2], y[3]) << 16,
                                                                      pack_e4m3(y[4], y[5]) | pack_e4m3(y[6], y[7]) << 16);
                } else {
                    o[i[q]] = uint8_t(pack_e4m3(y[0], 0.0f));
                }
            }
    } else {
        uint16_t *o = static_cast<uint16_t *>(a.out) + r * a.out_stride;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (i[q] < a.dim) {
                float y[W];
#pragma unroll
                for (int j = 0; j < W; ++j) y[j] = h[q][j] * w[q][j] * rs;
                if constexpr (VEC) {
                    *reinterpret_cast<uint4 *>(o + i[q]) =
                        make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
                } else {
                    store1<false>(o, i[q], y[0]);
                }
            }
    }
}

template <int E, bool VEC, bool XF, int DF, bool E4M3>
int run(const NormArgs &a, int threads, void *stream) {
    return launch_step(norm_kernel<E, VEC, XF, DF, E4M3>, int(a.rows), threads, 0, 1, stream, a);
}

template <int E, bool VEC, bool XF, int DF>
int pick_out(const NormArgs &a, bool e4m3, int threads, void *stream) {
    return e4m3 ? run<E, VEC, XF, DF, true>(a, threads, stream) : run<E, VEC, XF, DF, false>(a, threads, stream);
}

template <int E, bool VEC, bool XF>
int pick_delta(const NormArgs &a, int delta_dtype, bool e4m3, int threads, void *stream) {
    if (delta_dtype < 0) return pick_out<E, VEC, XF, -1>(a, e4m3, threads, stream);
    return delta_dtype == W12_F32 ? pick_out<E, VEC, XF, 1>(a, e4m3, threads, stream)
                                  : pick_out<E, VEC, XF, 0>(a, e4m3, threads, stream);
}

template <int E, bool VEC>
int pick(const NormArgs &a, int x_dtype, int delta_dtype, bool e4m3, int threads, void *stream) {
    return x_dtype == W12_F32 ? pick_delta<E, VEC, true>(a, delta_dtype, e4m3, threads, stream)
                              : pick_delta<E, VEC, false>(a, delta_dtype, e4m3, threads, stream);
}

}  // namespace

int launch_norm(const NormArgs &a, int x_dtype, int delta_dtype, int out_dtype, bool vec, void *stream) {
    const bool e4m3 = out_dtype == W12_E4M3;
    const auto threads = [&](int e) { return ((a.dim + e - 1) / e + 31) / 32 * 32; };
    if (vec) {
        if (threads(8) <= 1024) return pick<8, true>(a, x_dtype, delta_dtype, e4m3, threads(8), stream);
        return pick<32, true>(a, x_dtype, delta_dtype, e4m3, threads(32), stream);
    }
    if (threads(8) <= 1024) return pick<8, false>(a, x_dtype, delta_dtype, e4m3, threads(8), stream);
    return pick<32, false>(a, x_dtype, delta_dtype, e4m3, threads(32), stream);
}

}  // namespace w12
