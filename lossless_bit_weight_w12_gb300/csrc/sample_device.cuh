// sample_device.cuh -- a row of logits as whole-number weights, shared by the
// sampling kernel (kernels_sample.cu) and the sampled verification
// (kernels_cut.cu, kernels_accept.cu).
#pragma once

#include <cstdint>

#include "device_common.cuh"

namespace w12 {

using u64 = unsigned long long;

constexpr float kOne31 = 2147483648.0f;

__device__ __forceinline__ u64 umax64(u64 a, u64 b) { return a > b ? a : b; }

// acc + w, in one instruction
__device__ __forceinline__ u64 add_wide(u64 acc, uint32_t w) {
    u64 r;
    asm("mad.wide.u32 %0, %1, 1, %2;" : "=l"(r) : "r"(w), "l"(acc));
    return r;
}

__device__ __forceinline__ u64 warp_sum64(u64 x) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}
__device__ __forceinline__ u64 warp_max64(u64 x) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x = umax64(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    return x;
}
__device__ __forceinline__ u64 warp_scan64(u64 x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 z = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += z;
    }
    return x;
}

// Bins of weights, largest first: 64 per octave of [1, 2^31].
__device__ __forceinline__ int weight_bin(uint32_t w) {
    return int(((158u << 23) - __float_as_uint(__uint2float_rz(w))) >> 17);
}

template <int DT>
struct Row {
    const void *x;      // this CTA's chunk (shared or global memory)
    const uint32_t *w;  // its weights, once they are kept (shared memory), or NULL
    int n;              // logits in it
    int i0, i1;         // this thread's
    bool vec;           // four at a time: the chunk starts on a 16- (bf16: 8-) byte boundary
    bool inf;           // the largest is +infinity: such logits count as 0, the others as -infinity
    uint32_t first;     // index of its first
    float mx, inv_t;

    __device__ __forceinline__ float clean(float v) const {
        if (inf) return v == INFINITY ? 0.0f : -INFINITY;
        return fmaxf(v, -INFINITY);  // NaN is never sampled
    }
    __device__ __forceinline__ float at(int i) const {
        return clean(DT == W12_F32 ? static_cast<const float *>(x)[i]
                                   : bf16_bits_to_float(static_cast<const uint16_t *>(x)[i]));
    }
    // logits i .. i + 3 (-infinity past the chunk); i is a multiple of 4
    __device__ __forceinline__ void at4(int i, float (&v)[4]) const {
        if (vec && i + 4 <= n) {
            if (DT == W12_F32) {
                const float4 f = reinterpret_cast<const float4 *>(x)[i >> 2];
                v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
            } else {
                const uint2 f = reinterpret_cast<const uint2 *>(x)[i >> 2];
                v[0] = bf16_bits_to_float(f.x & 0xFFFFu), v[1] = bf16_bits_to_float(f.x >> 16);
                v[2] = bf16_bits_to_float(f.y & 0xFFFFu), v[3] = bf16_bits_to_float(f.y >> 16);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = clean(v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = i + j < n ? at(i + j) : -INFINITY;
        }
    }
    __device__ __forceinline__ u64 comp(float v, int i) const { return pack_key(v, first + uint32_t(i)); }
    // (max - x) / t as the exponent's argument, <= 0
    __device__ __forceinline__ float arg(float v) const { return __fmul_rn(__fsub_rn(v, mx), inv_t); }
    // (an argument of -infinity, or NaN -- an infinity times 0 -- gives 0)
    __device__ __forceinline__ uint32_t weight(float v) const { return __float2uint_rn(expf(arg(v)) * kOne31); }
    __device__ __forceinline__ uint32_t weight_at(int i) const { return w ? w[i] : weight(at(i)); }
    __device__ __forceinline__ void weight4(int i, uint32_t (&y)[4]) const {
        if (w) {  // (kept up to a multiple of 4)
            const uint4 f = reinterpret_cast<const uint4 *>(w)[i >> 2];
            y[0] = f.x, y[1] = f.y, y[2] = f.z, y[3] = f.w;
        } else {
            float v[4];
            at4(i, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = weight(v[j]);
        }
    }
};

// floor(u total / 2^24) with u in [0, 2^24)
__device__ __forceinline__ u64 scaled(uint64_t u, u64 total) { return (__umul64hi(u, total) << 40) | ((u * total) >> 24); }

__device__ __forceinline__ uint64_t fixed_u(float u) {
    const float f = u * 16777216.0f;
    return f >= 16777215.0f ? 16777215ull : f > 0.0f ? uint64_t(f) : 0ull;
}

// ceil(p total), at least 1: what lies before a token that stays
__device__ __forceinline__ u64 nucleus(uint64_t p, u64 total) {
    const u64 lim = p * (total >> 24) + ((p * (total & 0xFFFFFFull) + 0xFFFFFFull) >> 24);
    return lim < 1 ? 1 : lim;
}

}  // namespace w12
