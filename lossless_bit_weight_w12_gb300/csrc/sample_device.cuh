// sample_device.cuh -- 64-bit sums and the arithmetic of whole-number weights, shared by
// the sampling kernel (kernels_sample.cu) and the sampled verification (kernels_cut.cu,
// kernels_accept.cu).
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
