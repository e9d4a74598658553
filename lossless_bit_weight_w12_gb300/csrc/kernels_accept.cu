// kernels_accept.cu -- verification of sampled drafts against the target's
// probabilities: the acceptance of each drafted token and the draw of the next
// one, from what the cuts leave of every row (RowCut).
//
// With p and q the target's and the drafter's probabilities after their cuts
// (whole-number weights times the reciprocal of their sum, in fp32), draft d
// stays iff u q(d) < p(d).  The next token comes from max(p - q, 0) at the first
// draft that does not stay -- which makes the tokens the target's own samples --
// or from p after the last one, or where there was no draft.  The differences
// are whole numbers again, round(2^44 (p - q)), so their sums and the draw do not
// depend on how the row is cut.
//
// A cluster per request.  Every CTA finds the first draft that does not stay (a
// thread per position), then the row's two distributions are read in pieces of
// consecutive tokens, one per warp of the cluster, and added up; the warp that
// holds the drawn token reads its piece again.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "draft_internal.h"
#include "sample_device.cuh"
#include "step_device.cuh"

namespace w12 {

namespace {

namespace cg = cooperative_groups;

constexpr int kAT = 512;  // threads per CTA
constexpr int kAW = kAT / 32;
constexpr int kMostCluster = 8;
constexpr float kOne44 = 17592186044416.0f;

// A row and what its cuts leave.
struct Dist {
    const void *x;
    int f32;
    RowCut c;
    float inv;  // 1 / total (0: no token stays)

    __device__ __forceinline__ void init(const void *logits, int is_f32, int64_t row, int64_t V, const RowCut *cuts) {
        x = static_cast<const unsigned char *>(logits) + row * V * (is_f32 ? 4 : 2);
        f32 = is_f32;
        c = cuts[row];
        inv = c.total ? __fdiv_rn(1.0f, __ull2float_rn(c.total)) : 0.0f;
    }
    __device__ __forceinline__ float logit(int64_t i) const {
        const float v = f32 ? __ldg(static_cast<const float *>(x) + i)
                            : bf16_bits_to_float(__ldg(static_cast<const uint16_t *>(x) + i));
        return c.inf ? (v == INFINITY ? 0.0f : -INFINITY) : fmaxf(v, -INFINITY);
    }
    // token i's weight among those that stay
    __device__ __forceinline__ uint32_t weight(int64_t i) const {
        if (c.total == 0) return 0u;
        if (c.one >= 0) return i == c.one ? 0x80000000u : 0u;
        const float v = logit(i);
        const uint32_t w = __float2uint_rn(expf(__fmul_rn(__fsub_rn(v, c.mx), c.inv_t)) * kOne31);
        if (w < c.w_thr || w < c.floor_w || (w == c.w_thr && c.thr && pack_key(v, uint32_t(i)) < c.thr)) return 0u;
        return w;
    }
    __device__ __forceinline__ float share(int64_t i) const { return __fmul_rn(__uint2float_rn(weight(i)), inv); }
};

__device__ __forceinline__ u64 above(float p, float q) {
    const float d = __fsub_rn(p, q);
    return d > 0.0f ? __float2ull_rn(d * kOne44) : 0ull;
}

__global__ void __launch_bounds__(kAT) accept_kernel(const __grid_constant__ AcceptArgs a) {
    cg::cluster_group cl = cg::this_cluster();
    __shared__ u64 s_warp[kAW], s_cta[2][kMostCluster];
    __shared__ int64_t s_first;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cs = int(cl.num_blocks()), me = int(cl.block_rank());
    const int64_t r = int64_t(blockIdx.x) / cs, drafts = a.T - 1;
    if (tid == 0) s_first = drafts;
    pdl_launch_dependents();
    cl.sync();  // another CTA's shared memory may be touched only once that CTA runs
    pdl_wait_previous();

    // ---- the first draft that does not stay
    for (int64_t i = tid; i < drafts; i += kAT) {
        const int64_t d = a.draft[r * drafts + i];
        float p = 0.0f, q = 0.0f;
        if (d >= 0 && d < a.V) {
            Dist x;
            x.init(a.logits, a.f32, r * a.T + i, a.V, a.cuts);
            p = x.share(d);
            x.init(a.draft_logits, a.draft_f32, r * drafts + i, a.V, a.draft_cuts);
            q = x.share(d);
        }
        if (a.ratio && me == 0) a.ratio[r * drafts + i] = p >= q ? (p > 0.0f ? 1.0f : 0.0f) : __fdiv_rn(p, q);
        if (!(__fmul_rn(a.u[r * a.T + i], q) < p)) atomicMin(reinterpret_cast<long long *>(&s_first), static_cast<long long>(i));
    }
    __syncthreads();
    const int64_t n = s_first;
    const bool none = n == drafts || a.draft[r * drafts + n] < 0 || a.draft[r * drafts + n] >= a.V;

    // ---- the next token
    Dist p, q;
    p.init(a.logits, a.f32, r * a.T + n, a.V, a.cuts);
    if (!none) q.init(a.draft_logits, a.draft_f32, r * drafts + n, a.V, a.draft_cuts);
    const int64_t each = ((a.V + cs * kAW - 1) / (cs * kAW) + 31) / 32 * 32;  // tokens per warp of the cluster
    const int64_t i0 = min(int64_t(me * kAW + warp) * each, a.V), i1 = min(i0 + each, a.V);
    bool rest = !none;
    for (int pass = 0; pass < 2; ++pass) {  // a second one where p - q leaves nothing
        const auto value = [&](int64_t i) -> u64 { return rest ? above(p.share(i), q.share(i)) : u64(p.weight(i)); };
        u64 mine = 0;
        for (int64_t i = i0 + lane; i < i1; i += 32) mine += value(i);
        mine = warp_sum64(mine);
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        if (tid < cs) {
            u64 s = 0;
            for (int w = 0; w < kAW; ++w) s += s_warp[w];
            cl.map_shared_rank(&s_cta[pass][0], tid)[me] = s;
        }
        cl.sync();
        u64 total = 0, before = 0;
        for (int c = 0; c < cs; ++c) {
            if (c < me) before += s_cta[pass][c];
            total += s_cta[pass][c];
        }
        for (int w = 0; w < warp; ++w) before += s_warp[w];
        if (total == 0) {
            if (rest) {
                rest = false;
                __syncthreads();
                continue;
            }
            if (me == 0 && tid == 0) a.accept_len[r] = int32_t(n), a.next_tok[r] = -1;
            break;
        }
        const u64 target = scaled(fixed_u(a.u[r * a.T + drafts]), total);
        if (before <= target && target < before + mine) {  // one warp of the cluster
            for (int64_t j = i0; j < i1; j += 32) {
                const u64 incl = warp_scan64(j + lane < i1 ? value(j + lane) : 0ull, lane);
                const uint32_t at = __ballot_sync(0xFFFFFFFFu, before + incl > target);
                if (at) {
                    if (lane == 0) a.accept_len[r] = int32_t(n), a.next_tok[r] = int32_t(j + __ffs(at) - 1);
                    break;
                }
                before += __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
        }
        break;
    }
    cl.sync();  // no CTA leaves while another may write its shared memory
}

}  // namespace

int launch_accept(const AcceptArgs &a, void *stream) {
    int cs = 1;
    while (cs < kMostCluster && a.V > int64_t(cs) * 4096) cs *= 2;
    return launch_step(accept_kernel, int(a.R * cs), kAT, 0, cs, stream, a);
}

}  // namespace w12
