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
// A request's row is cut into pieces of consecutive tokens, one per CTA.  Every CTA
// finds the first draft that does not stay (a thread per position; the drafts' shares
// of p and q come with the cuts), and each of its warps adds a run of its piece up;
// the last CTA to finish finds the run that holds the drawn token and goes through
// that again.
//
// What bounds it: the instructions of two exact exponentials a token (some 115 in all
// where nothing is cut, so few requests are spread over all SMs; where tokens are cut, a
// warp passes over fours without one that stays), and the steps that wait for one
// another: 16 requests of 151936 tokens 18 us of 65, of which the sums 9, the end 6.
// Loops are short on purpose: an SM that has not met a piece of code yet waits some
// 250 cycles per 128 bytes of it (sixteen tokens unrolled: 8 us of a single request's
// 17), and both passes go through one loop for the same reason.  Two tokens a turn: 16
// x 8 rows 65 us in all; one 68, four 66.
#include <cuda_runtime.h>

#include <algorithm>

#include "cut_device.cuh"
#include "draft_internal.h"
#include "step_device.cuh"

namespace w12 {

namespace {

constexpr int kAT = 256;        // threads per CTA
constexpr int kAW = kAT / 32;
static_assert(kAW == kAcceptRuns, "a run a warp");
constexpr int kStep = 4 * kAT;  // tokens of a CTA at a time
constexpr float kOne44 = 17592186044416.0f;

// A row and what its cuts leave.  (The logits are read from L2, here as in the kernel
// ahead: the read-only path is not for memory that was written after this kernel began.)
struct Dist {
    const void *x;
    int f32, vec;
    RowCut c;

    __device__ __forceinline__ void init(const void *logits, int is_f32, int64_t row, int64_t V, const RowCut *cuts) {
        x = static_cast<const unsigned char *>(logits) + row * V * (is_f32 ? 4 : 2);
        f32 = is_f32, vec = (reinterpret_cast<uintptr_t>(x) & (is_f32 ? 15 : 7)) == 0;
        c = cuts[row];
    }
    __device__ __forceinline__ uint32_t bits(int i) const {
        return f32 ? __float_as_uint(__ldcg(static_cast<const float *>(x) + i)) : uint32_t(__ldcg(static_cast<const uint16_t *>(x) + i));
    }
    // Logits i .. i + 3 as they lie in memory (i a multiple of 4; from `end` on:
    // -infinity), so that nothing waits for them before they are used.
    __device__ __forceinline__ uint4 read(int i, int end) const {
        uint4 r = make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
        if (!f32) r.x = r.y = 0xFF80FF80u;
        if (i + 4 <= end && vec) {
            if (f32) {
                r = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const float *>(x) + i));
            } else {
                const uint2 y = __ldcg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(x) + i));
                r.x = y.x, r.y = y.y;
            }
        } else if (i < end) {
            const uint32_t none = f32 ? 0xFF800000u : 0xFF80u;
            const uint32_t b0 = bits(i), b1 = i + 1 < end ? bits(i + 1) : none, b2 = i + 2 < end ? bits(i + 2) : none;
            const uint32_t b3 = i + 3 < end ? bits(i + 3) : none;
            r = f32 ? make_uint4(b0, b1, b2, b3) : make_uint4(b0 | b1 << 16, b2 | b3 << 16, 0u, 0u);
        }
        return r;
    }
    // The same for a row of which one token stays: that one's logit need not be read.
    __device__ __forceinline__ uint4 read_one(int i) const {
        const uint32_t none = 0xFF800000u, top = __float_as_uint(c.least);
        const int k = c.one - i;
        const uint4 r = make_uint4(k == 0 ? top : none, k == 1 ? top : none, k == 2 ? top : none, k == 3 ? top : none);
        return f32 ? r : make_uint4(r.x >> 16 | (r.y & 0xFFFF0000u), r.z >> 16 | (r.w & 0xFFFF0000u), 0u, 0u);
    }
    __device__ __forceinline__ float4 floats(const uint4 &r) const {
        return f32 ? make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w))
                   : make_float4(bf16_bits_to_float(r.x & 0xFFFFu), __uint_as_float(r.x & 0xFFFF0000u),
                                 bf16_bits_to_float(r.y & 0xFFFFu), __uint_as_float(r.y & 0xFFFF0000u));
    }
};

// round(2^44 max(p - q, 0)): below 2^31 in one conversion, else 20 bits and the 24
// below them, which are exact in the float's remainder.
__device__ __forceinline__ u64 above(float p, float q) {
    const float d = __fsub_rn(p, q);
    if (!(d > 0.0f)) return 0ull;
    const float y = d * kOne44;
    if (y < 2147483648.0f) return u64(__float2uint_rn(y));
    const float z = d * 1048576.0f;
    const uint32_t hi = __float2uint_rz(z);
    return (u64(hi) << 24) + u64(__float2uint_rn((z - __uint2float_rn(hi)) * 16777216.0f));
}

// What a request's CTAs share: the row that is drawn from, and, where a draft was
// refused (rest), the drafter's.
struct Draw {
    Dist p, q;
    int rest;
};

// The sum over the block, and what lies before this thread.
__device__ __forceinline__ u64 block_scan(u64 *s_warp, u64 mine, u64 *before) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const u64 incl = warp_scan64(mine, lane);
    __syncthreads();
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    u64 total = 0, b = incl - mine;
#pragma unroll
    for (int w = 0; w < kAW; ++w) {
        if (w < warp) b += s_warp[w];
        total += s_warp[w];
    }
    *before = b;
    return total;
}

__global__ void __launch_bounds__(kAT, 4) accept_kernel(const __grid_constant__ AcceptArgs a) {
    __shared__ u64 s_warp[kAW];
    __shared__ long long s_first;
    __shared__ Draw d;
    __shared__ int s_last, s_run;
    __shared__ u64 s_left;  // what is left of the drawn number at the run
    __shared__ u64 s_each[4 * kAT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t r = int64_t(blockIdx.x) / a.pieces, drafts = a.T - 1;
    const int me = int(blockIdx.x % a.pieces), V = int(a.V);
    if (tid == 0) s_first = drafts;
    pdl_launch_dependents();
    pdl_wait_previous();
    __syncthreads();

    // ---- the first draft that does not stay
#pragma unroll 1
    for (int64_t i = tid; i < drafts; i += kAT) {
        const float p = a.cuts[r * a.T + i].share, q = a.draft_cuts[r * drafts + i].share;
        if (!(__fmul_rn(a.u[r * a.T + i], q) < p)) atomicMin(&s_first, static_cast<long long>(i));
        if (a.ratio && me == 0) a.ratio[r * drafts + i] = p >= q ? (p > 0.0f ? 1.0f : 0.0f) : __fdiv_rn(p, q);
    }
    __syncthreads();
    const int64_t n = s_first;
    if (tid == 0) d.p.init(a.logits, a.f32, r * a.T + n, a.V, a.cuts);
    if (tid == 32) {
        const int64_t t = n < drafts ? a.draft[r * drafts + n] : -1;
        d.rest = t >= 0 && t < a.V;
        if (d.rest) d.q.init(a.draft_logits, a.draft_f32, r * drafts + n, a.V, a.draft_cuts);
    }
    __syncthreads();

    const int refused = d.rest;
    const auto read_y = [&](int i, int end) {
        return !refused ? make_uint4(0u, 0u, 0u, 0u) : d.q.c.one < 0 ? d.q.read(i, end) : d.q.read_one(i);
    };
    // ---- pass 0: the sums of this warp's run of tokens; pass 1, in the last CTA: the
    // run that holds the drawn token once more, all threads on it (one loop for both,
    // so that its code is there when the second begins)
    const int run = a.each / kAW, runs = a.pieces * kAW;
    ulonglong2 *part = a.parts + r * runs;
    const RowCut pc = d.p.c, qc = d.q.c;
    int rest = refused, hop = 128, trips = run / 128;
    int i = me * a.each + warp * run + 4 * lane, end = min(me * a.each + (warp + 1) * run, V);
    u64 left = 0;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        u64 sum_rest = 0, sum_own = 0;
        uint4 x0 = d.p.read(i, end), y0 = read_y(i, end), x1 = d.p.read(i + hop, end), y1 = read_y(i + hop, end);
#pragma unroll 1
        for (int k = 0; k < trips; ++k, i += hop) {
            const uint4 x2 = d.p.read(i + 2 * hop, end), y2 = read_y(i + 2 * hop, end);
            float4 x = d.p.floats(x0);
            x0 = x1, x1 = x2;
            u64 here = 0;
            // (cut rows: most tokens are below)
            int j = __any_sync(0xFFFFFFFFu, fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)) >= pc.least) || pass ? 0 : 4;
            float4 y = d.q.floats(y0);
            y0 = y1, y1 = y2;
#pragma unroll 1
            for (; j < 4; j += 2, x.x = x.z, x.y = x.w, y.x = y.z, y.y = y.w) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const Weight w = cut_weight(pc, e ? x.y : x.x, i + j + e);
                    u64 z = 0;
                    sum_own = add_wide(sum_own, w.whole);
                    if (refused) {
                        z = above(__fmul_rn(w.f, pc.inv), __fmul_rn(cut_weight(qc, e ? y.y : y.x, i + j + e).f, qc.inv));
                        sum_rest += z;
                    }
                    if (pass) {
                        if (!rest) z = w.whole;
                        s_each[4 * tid + j + e] = z;
                        here += z;
                    }
                }
            }
            if (pass == 0) continue;
            u64 before;
            const u64 all = block_scan(s_warp, here, &before);
            if (left < all) {
                if (before <= left && left < before + here) {
                    left -= before;
                    int j = 0;
#pragma unroll 1
                    for (; j < 3 && left >= s_each[4 * tid + j]; ++j) left -= s_each[4 * tid + j];
                    a.accept_len[r] = int32_t(n), a.next_tok[r] = i + j;
                }
                return;
            }
            left -= all;
        }
        if (pass) return;  // (not reached: the run holds it)
        sum_rest = warp_sum64(sum_rest), sum_own = warp_sum64(sum_own);
        if (lane == 0) __stcg(&part[me * kAW + warp], make_ulonglong2(sum_rest, sum_own));
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            s_last = atomicAdd(&a.arrived[r], 1u) == uint32_t(a.pieces - 1);
        }
        __syncthreads();
        if (!s_last) return;
        __threadfence();
        const int per = (runs + kAT - 1) / kAT, c0 = min(tid * per, runs), c1 = min(c0 + per, runs);
        u64 total, mine, before;
#pragma unroll 1
        for (;; rest = 0) {  // (where p - q leaves nothing: p)
            mine = 0;
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
                const ulonglong2 z = __ldcg(&part[c]);
                mine += rest ? z.x : z.y;
            }
            total = block_scan(s_warp, mine, &before);
            if (total || !rest) break;
        }
        if (total == 0) {
            if (tid == 0) a.accept_len[r] = int32_t(n), a.next_tok[r] = -1;
            return;
        }
        const u64 target = scaled(fixed_u(a.u[r * a.T + drafts]), total);
        if (before <= target && target < before + mine) {
            left = target - before;
            int c = c0;
#pragma unroll 1
            for (; c + 1 < c1; ++c) {
                const ulonglong2 z = __ldcg(&part[c]);
                if (left < (rest ? z.x : z.y)) break;
                left -= rest ? z.x : z.y;
            }
            s_run = c, s_left = left;
        }
        __syncthreads();
        left = s_left;
        i = s_run * run + 4 * tid, end = min((s_run + 1) * run, V), hop = 4 * kAT, trips = (run + 4 * kAT - 1) / (4 * kAT);
    }
}

}  // namespace

// Pieces of whole steps, as many as fill the GPU (four CTAs on each of 152 SMs).
void accept_pieces(int64_t R, int64_t V, int32_t *each, int32_t *pieces) {
    const int64_t steps = (V + kStep - 1) / kStep;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(steps, 608 / R));
    const int64_t per = (steps + want - 1) / want;
    *each = int32_t(per * kStep);
    *pieces = int32_t((steps + per - 1) / per);
}

int launch_accept(const AcceptArgs &a, void *stream) {
    return launch_step(accept_kernel, int(a.R * a.pieces), kAT, 0, 1, stream, a);
}

}  // namespace w12
