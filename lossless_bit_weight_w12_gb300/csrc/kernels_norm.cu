// kernels_norm.cu -- residual addition and root-mean-square norm of rows, out
// in bf16 or in e4m3 with one fp32 scale per row.
//
//   h = x + delta,  r = 1 / sqrt(mean(h^2) + eps),  y = (h (weight + offset)) r
//
// A CTA takes a row at a time, in registers: every tensor is read or written once.
// It asks for its next row before it reduces the one it has, so that the memory is
// busy under the reductions; the weights stay in registers from row to row.  What
// bounds it: from some hundred rows on the memory (8187 rows of 5120, bf16 with delta
// and residual: 335 MB in 53 us, 93 % of the copy rate; asked for after the reductions
// 62), below that the launch (one row 7.4 us with the host's call).  Wider elements leave
// fewer rows under way in 40 registers a thread, which nearly every form passes (-Xptxas
// -v: bf16 4 bytes of spills, fp32 with fp32 delta to e4m3 some 130): 8187 x 5120 with
// residual, fp32 and fp32 delta to bf16 96 us (86 for the bytes), to e4m3 114 (80), bf16
// and fp32 delta to e4m3 81 (56).  Past 8192 elements a row has no next one under it and
// the weights are read again: 4096 x 16384 bf16 111 us (79).  A call with any tensor off
// 16-byte boundaries, or dim no multiple of 8, goes one element at a time throughout:
// 3001 rows of 2883 fp32 elements 24 us, 70 % of the copy rate.
//
// The e4m3 scale needs the largest |y|; as r is one positive number for the
// row and a rounded product does not decrease with its factor, it is the
// rounded product of r and the largest |h (weight + offset)|, so one block
// reduction carries both the sum of squares and that maximum (as the bits of
// |.|, which order like the numbers and put NaN above infinity).
//
// The sum of squares is fp32.  Where it (or with eps the mean) overflows, the row is
// scaled by 2^-80 in its registers and reduced once more, with eps times 2^-160.
// Where it is so small that squares underflow and eps does not outweigh them, the
// row is scaled by 2^50, up to three times (a row of fp32's smallest numbers ends
// at 2^1); powers of two round nothing, and at 2^0 the largest scaled row leaves
// the weights 2^120.
#include <cuda_runtime.h>

#include <algorithm>

#include "device_common.cuh"
#include "draft_internal.h"
#include "step_device.cuh"

namespace w12 {

namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyRow = 1e-30f;
constexpr float kTinySquare = 0x1p-100f;  // mean squares below it: the squares' own roundings (2^-150) count
constexpr float kTinyEps = 0x1p-40f;      // from here on eps outweighs them

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

// Elements of a row as they lie in memory: eight consecutive ones, or one.
template <bool VEC, bool F32>
struct Raw {
    uint4 v[VEC ? (F32 ? 2 : 1) : 1];  // (one element: in v[0].x)

    __device__ __forceinline__ void load(const void *row, int i) {
        if constexpr (VEC) {
            const unsigned char *p = static_cast<const unsigned char *>(row) + size_t(i) * (F32 ? 4 : 2);
            v[0] = load16(p);
            if constexpr (F32) v[1] = load16(p + 16);
        } else {
            v[0].x = F32 ? __float_as_uint(static_cast<const volatile float *>(row)[i])
                         : uint32_t(static_cast<const volatile uint16_t *>(row)[i]) << 16;
        }
    }
    __device__ __forceinline__ void get(float (&f)[VEC ? 8 : 1]) const {
        if constexpr (!VEC) {
            f[0] = __uint_as_float(v[0].x);
        } else if constexpr (F32) {
            f[0] = __uint_as_float(v[0].x), f[1] = __uint_as_float(v[0].y), f[2] = __uint_as_float(v[0].z), f[3] = __uint_as_float(v[0].w);
            f[4] = __uint_as_float(v[1].x), f[5] = __uint_as_float(v[1].y), f[6] = __uint_as_float(v[1].z), f[7] = __uint_as_float(v[1].w);
        } else {
            f[0] = bf_lo(v[0].x), f[1] = bf_hi(v[0].x), f[2] = bf_lo(v[0].y), f[3] = bf_hi(v[0].y);
            f[4] = bf_lo(v[0].z), f[5] = bf_hi(v[0].z), f[6] = bf_lo(v[0].w), f[7] = bf_hi(v[0].w);
        }
    }
};

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
// T: threads at most (768: two CTAs of them on an SM, with 40 registers a thread).
template <int E, bool VEC, bool XF, int DF, bool E4M3, int T>
__global__ void __launch_bounds__(T, 1536 / T) norm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float s_sum[4][32];
    __shared__ uint32_t s_top[4][32];
    const int tid = threadIdx.x, step = blockDim.x;
    constexpr int W = VEC ? 8 : 1, Q = E / W;
    pdl_launch_dependents();
    pdl_wait_previous();
    const auto at = [](const void *p, int64_t elements, bool f32) {
        return static_cast<const unsigned char *>(p) + elements * (f32 ? 4 : 2);
    };
    constexpr bool kAhead = E == 8;  // (32 elements a thread leave no registers for a second row, or for weights)
    int i[Q];
    Raw<VEC, XF> x[kAhead ? Q : 1];
    Raw<VEC, (DF > 0)> d[kAhead ? Q : 1];
    const auto ask = [&](int64_t r, int q, int to) {
        if (i[q] >= a.dim) return;
        x[to].load(at(a.x, r * a.x_stride, XF), i[q]);
        if constexpr (DF >= 0) d[to].load(at(a.delta, r * a.delta_stride, DF > 0), i[q]);
    };
    const auto load_weights = [&](int q, float(&w)[W]) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = 1.0f;
        if (a.weight && i[q] < a.dim) {
            if (a.weight_f32) {
                Raw<VEC, true> y;
                y.load(a.weight, i[q]);
                y.get(w);
            } else {
                Raw<VEC, false> y;
                y.load(a.weight, i[q]);
                y.get(w);
            }
        }
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] += a.offset;
    };
#pragma unroll
    for (int q = 0; q < Q; ++q) i[q] = (tid + q * step) * W;
    int64_t r = blockIdx.x;
    float kept[kAhead ? Q : 1][W];
    if constexpr (kAhead) {
#pragma unroll
        for (int q = 0; q < Q; ++q) ask(r, q, q);
#pragma unroll
        for (int q = 0; q < Q; ++q) load_weights(q, kept[q]);
    }
    const auto weights = [&](int q, float(&w)[W]) {
        if constexpr (kAhead) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j] = kept[q][j];
        } else {
            load_weights(q, w);
        }
    };
    int buffer = 0;  // (a buffer of the reduction is used again two rows later)
    for (; r < a.rows; r += gridDim.x, buffer ^= 2) {
        float h[Q][W];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if constexpr (!kAhead) ask(r, q, 0);
            if (i[q] < a.dim) {
                x[kAhead ? q : 0].get(h[q]);
                if constexpr (DF >= 0) {
                    float y[W];
                    d[kAhead ? q : 0].get(y);
#pragma unroll
                    for (int j = 0; j < W; ++j) h[q][j] += y[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) h[q][j] = 0.0f;
            }
        }
        if constexpr (kAhead)  // (the residual, written below, may be x: other rows of it)
            if (r + gridDim.x < a.rows)
#pragma unroll
                for (int q = 0; q < Q; ++q) ask(r + gridDim.x, q, q);
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
            for (int q = 0; q < Q; ++q) {
                float w[W];
                if (E4M3) weights(q, w);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    sum = fmaf(h[q][j], h[q][j], sum);
                    if (E4M3) top = max(top, __float_as_uint(h[q][j] * w[j]) & 0x7FFFFFFFu);
                }
            }
            // (two buffers in turn: a barrier lies between a buffer's last read and its next write)
            reduce(sum, top, s_sum[buffer + (pass & 1)], s_top[buffer + (pass & 1)]);
            const bool large = pass == 0 && (sum == INFINITY || (eps > 0x1p100f && sum > (0x1p127f - eps) * float(a.dim)));
            const bool small = pass < 3 && eps < kTinyEps && sum < kTinySquare * float(a.dim);
            if (!large && !small) break;
            const float by = large ? 0x1p-80f : 0x1p50f;
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int j = 0; j < W; ++j) h[q][j] *= by;
            eps = eps * by * by;
        }
        const float ms = __fdiv_rn(sum, float(a.dim)) + eps;
        const float rs = ms == 0.0f ? 0.0f : __fdiv_rn(1.0f, __fsqrt_rn(ms));  // (0: a row of zeros, and eps 0)
        if constexpr (E4M3) {
            const float amax = __uint_as_float(top) * rs;
            const bool bad = !(amax <= 3.402823466e38f), some = amax > kTinyRow;
            const float inv = !bad && some ? __fdiv_rn(kE4m3Max, amax) : 0.0f;
            if (tid == 0) a.scale[r] = bad ? __uint_as_float(0x7FC00000u) : some ? __fdiv_rn(amax, kE4m3Max) : 0.0f;
            uint8_t *o = static_cast<uint8_t *>(a.out) + r * a.out_stride;
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (i[q] < a.dim) {
                    float y[W], w[W];
                    weights(q, w);
                    // (inv 0: zeros, also where the row holds a NaN or an infinity)
#pragma unroll
                    for (int j = 0; j < W; ++j) y[j] = inv > 0.0f ? h[q][j] * w[j] * rs * inv : 0.0f;
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
                    float y[W], w[W];
                    weights(q, w);
#pragma unroll
                    for (int j = 0; j < W; ++j) y[j] = h[q][j] * w[j] * rs;
                    if constexpr (VEC) {
                        *reinterpret_cast<uint4 *>(o + i[q]) =
                            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
                    } else {
                        store1<false>(o, i[q], y[0]);
                    }
                }
        }
    }
}

// As many CTAs as fit on the GPU at a time (1536 threads an SM with 40 registers each,
// for elements by eights, else 1024 with 64).
template <int E, bool VEC, bool XF, int DF, bool E4M3>
int run(const NormArgs &a, int threads, void *stream) {
    const auto grid = [&](int per_sm) { return int(std::min(a.rows, int64_t(a.sms) * std::max(1, per_sm / threads))); };
    if constexpr (E == 8 && VEC)
        if (threads <= 768)
            return launch_step(norm_kernel<E, VEC, XF, DF, E4M3, 768>, grid(1536), threads, 0, 1, stream, a);
    return launch_step(norm_kernel<E, VEC, XF, DF, E4M3, 1024>, grid(1024), threads, 0, 1, stream, a);
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
