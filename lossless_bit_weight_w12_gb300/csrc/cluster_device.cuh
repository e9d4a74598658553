// cluster_device.cuh -- barriers of a thread-block cluster.
#pragma once

namespace w12 {

// A cluster barrier at which only warp 0 has written for other CTAs (the
// others need not wait until their own writes have gone out).
__device__ __forceinline__ void sync_sums() {
    if (threadIdx.x < 32)
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    else
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// One that hands nothing over.
__device__ __forceinline__ void sync_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// One in two halves, for the cluster's start: another CTA's shared memory may be
// touched only once that CTA runs.
__device__ __forceinline__ void cluster_here() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

}  // namespace w12
