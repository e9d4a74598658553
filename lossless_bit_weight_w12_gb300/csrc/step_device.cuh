// step_device.cuh -- small device helpers of the decode-step kernels:
// dependent-launch control, bf16, fp16 and e4m3 conversions.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace w12 {

// Let the next kernel of the stream start its prologue; wait until the
// previous one has completed with its memory visible (no-ops for launches
// without the programmatic-serialization attribute).
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Two floats as a bf16 pair, nearest even, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two floats as an fp16 pair, nearest even, the first in the low half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes (the low 16 bits of w, or the high ones) as an fp16 pair:
// exact, every e4m3 value is an fp16 value.
__device__ __forceinline__ uint32_t e4m3x2_lo_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float (&f)[4]) {
    const uint32_t a = e4m3x2_lo_to_f16x2(w), b = e4m3x2_hi_to_f16x2(w);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    f[0] = x.x, f[1] = x.y, f[2] = y.x, f[3] = y.y;
}

}  // namespace w12
