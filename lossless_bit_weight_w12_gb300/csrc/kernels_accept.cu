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
// finds the first draft that does not stay (a thread per position) and adds its
// piece up; the last one to finish finds the piece that holds the drawn token and
// goes through it again.
//
// What bounds it: the instructions of two exact exponentials a token (some 50
// where nothing is cut, so few requests are spread over all SMs), and the steps
// that wait for one another.  Loops are rolled on purpose: an SM that has not met a
// piece of code yet waits some 250 cycles per 128 bytes of it (sixteen tokens
// unrolled: 8 us of a single request's 17).
#include <cuda_runtime.h>

#include <algorithm>

#include "draft_internal.h"
#include "sample_device.cuh"
#include "step_device.cuh"

namespace w12 {

namespace {

constexpr int kAT = 256;        // threads per CTA
constexpr int kAW = kAT / 32;
constexpr int kStep = 4 * kAT;  // tokens of a CTA at a time
constexpr float kOne44 = 17592186044416.0f;

// A row and what its cuts leave.
struct Dist {
    const void *x;
    int f32, vec;
    int easy;     // some token stays, and none is infinite
    int last;     // the highest index that stays among the logits of `least`
    RowCut c;
    float inv;    // 1 / total (0: no token stays)
    float least;  // the tokens that stay have logits from it on

    __device__ __forceinline__ void init(const void *logits, int is_f32, int64_t row, int64_t V, const RowCut *cuts) {
        x = static_cast<const unsigned char *>(logits) + row * V * (is_f32 ? 4 : 2);
        f32 = is_f32, vec = (reinterpret_cast<uintptr_t>(x) & (is_f32 ? 15 : 7)) == 0;
        c = cuts[row];
        inv = c.total ? __fdiv_rn(1.0f, __ull2float_rn(c.total)) : 0.0f;
        easy = c.total != 0 && !c.inf;
        last = c.one >= 0 ? c.one : c.thr ? int(key_index(c.thr)) : 0x7FFFFFFF;
        const uint32_t k = uint32_t(c.thr >> 32);
        const float at = __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
        least = c.total == 0 ? INFINITY : c.inf ? 0.0f : c.one >= 0 ? c.mx : c.thr ? at : -INFINITY;
    }
    // the weight of token i with logit v, of an easy row (a single token that stays is
    // the first of the largest: mx, with 1 / t as 1)
    __device__ __forceinline__ uint32_t easy_weight(float v, int i) const {
        const uint32_t w = __float2uint_rn(expf(__fmul_rn(__fsub_rn(v, c.mx), c.inv_t)) * kOne31);
        return (v > least || (v == least && i <= last)) && w >= c.floor_w ? w : 0u;
    }
    __device__ __forceinline__ float logit(int i) const {
        return f32 ? __ldg(static_cast<const float *>(x) + i)
                   : bf16_bits_to_float(__ldg(static_cast<const uint16_t *>(x) + i));
    }
    // logits i .. i + 3 (i a multiple of 4; past V: -infinity)
    __device__ __forceinline__ float4 logits4(int i, int V) const {
        if (i + 4 <= V && vec) {
            if (f32) return __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i));
            const uint2 y = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(x) + i));
            return make_float4(bf16_bits_to_float(y.x & 0xFFFFu), __uint_as_float(y.x & 0xFFFF0000u),
                               bf16_bits_to_float(y.y & 0xFFFFu), __uint_as_float(y.y & 0xFFFF0000u));
        }
        const auto at = [&](int j) { return i + j < V ? logit(i + j) : -INFINITY; };
        return make_float4(at(0), at(1), at(2), at(3));
    }
    // the weight of token i with logit v among those that stay (v past V: -infinity)
    __device__ __noinline__ uint32_t weight(float v, int i) const {
        if (c.one >= 0) return i == c.one ? 0x80000000u : 0u;
        if (!(v >= least)) return 0u;
        if (c.inf) v = v == INFINITY ? 0.0f : -INFINITY;
        const uint32_t w = __float2uint_rn(expf(__fmul_rn(__fsub_rn(v, c.mx), c.inv_t)) * kOne31);
        if (w < c.w_thr || w < c.floor_w) return 0u;
        if (w == c.w_thr && c.thr && pack_key(v, uint32_t(i)) < c.thr) return 0u;
        return w;
    }
    __device__ __forceinline__ float share(float v, int i) const { return __fmul_rn(__uint2float_rn(weight(v, i)), inv); }
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

// What a request's CTAs share: the row that is drawn from.
struct Draw {
    Dist p, q;
    int rest;  // from p - q
};

// The draw's weights of tokens i .. i + 3 (logits x and y): their sum, and in
// whole the target's own.  Where the sum -- of the target's own if !rest -- passes
// `stop`, *at is the token.
__device__ __forceinline__ u64 quad(const Draw &d, bool rest, int i, float4 x, float4 y, u64 &whole, u64 stop, int *at) {
    u64 sum = 0;
    const bool easy = d.p.easy && (!d.rest || d.q.easy);
    const float ip = d.p.inv, iq = d.q.inv, least = d.p.least;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
        if (!__any_sync(0xFFFFFFFFu, x.x >= least)) {
            // (cut rows: most of them)
        } else if (easy) {
            const uint32_t w = d.p.easy_weight(x.x, i + j), z = d.rest ? d.q.easy_weight(y.x, i + j) : 0u;
            whole = add_wide(whole, w);
            const u64 a = above(__fmul_rn(__uint2float_rn(w), ip), __fmul_rn(__uint2float_rn(z), iq));
            sum += rest ? a : u64(w);
        } else {
            const uint32_t w = d.p.weight(x.x, i + j);
            whole = add_wide(whole, w);
            if (!rest)
                sum += w;
            else if (w)
                sum += above(__fmul_rn(__uint2float_rn(w), ip), d.q.share(y.x, i + j));
        }
        if (sum > stop) {
            if (*at < 0) *at = i + j;
        }
        x = make_float4(x.y, x.z, x.w, 0.0f), y = make_float4(y.y, y.z, y.w, 0.0f);
    }
    return sum;
}

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
    __shared__ int s_last, s_piece, s_token;
    __shared__ u64 s_before;
    const int tid = threadIdx.x;
    const int64_t r = int64_t(blockIdx.x) / a.pieces, drafts = a.T - 1;
    const int me = int(blockIdx.x % a.pieces), V = int(a.V);
    if (tid == 0) s_first = drafts;
    pdl_launch_dependents();
    pdl_wait_previous();
    __syncthreads();

    // ---- the first draft that does not stay
#pragma unroll 1
    for (int64_t i = tid; i < drafts; i += kAT) {
        const int64_t t = a.draft[r * drafts + i];
        Dist x, y;
        x.init(a.logits, a.f32, r * a.T + i, a.V, a.cuts);
        y.init(a.draft_logits, a.draft_f32, r * drafts + i, a.V, a.draft_cuts);
        const bool there = t >= 0 && t < a.V;
        const float vx = there ? x.logit(int(t)) : 0.0f, vy = there ? y.logit(int(t)) : 0.0f;
        const float p = there ? x.share(vx, int(t)) : 0.0f, q = there ? y.share(vy, int(t)) : 0.0f;
        if (a.ratio && me == 0) a.ratio[r * drafts + i] = p >= q ? (p > 0.0f ? 1.0f : 0.0f) : __fdiv_rn(p, q);
        if (!(__fmul_rn(a.u[r * a.T + i], q) < p)) atomicMin(&s_first, static_cast<long long>(i));
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

    // ---- this piece's sums
    const bool read_q = d.rest && d.q.c.one < 0;
    const float4 none = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    const auto read_x = [&](int i, int end) { return i < end ? d.p.logits4(i, V) : none; };
    const auto read_y = [&](int i, int end) {
        if (read_q && i < end) return d.q.logits4(i, V);
        const int k = d.rest ? d.q.c.one - i : -1;  // (the one token's logit need not be read)
        const auto at = [&](int j) { return j == k ? d.q.c.mx : -INFINITY; };
        return make_float4(at(0), at(1), at(2), at(3));
    };
    u64 mine = 0, whole = 0, before;
    int at = 0;
    u64 *part = a.parts + (r * a.pieces) * 2;
    {
        const int end = min((me + 1) * a.each, V);
        int i = me * a.each + 4 * tid;
        float4 x = read_x(i, end), y = read_y(i, end);
#pragma unroll 1
        for (int i0 = me * a.each; i0 < end; i0 += kStep, i += kStep) {  // (the next ones are on their way)
            const float4 nx = read_x(i + kStep, end), ny = read_y(i + kStep, end);
            mine += quad(d, d.rest, i, x, y, whole, ~0ull, &at);
            x = nx, y = ny;
        }
    }
    mine = block_scan(s_warp, mine, &before);
    whole = block_scan(s_warp, whole, &before);
    if (tid == 0) {
        __stcg(&part[2 * me], mine);
        __stcg(&part[2 * me + 1], whole);
        __threadfence();
        s_last = atomicAdd(&a.arrived[r], 1u) == uint32_t(a.pieces - 1);
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();

    // ---- the last CTA: the piece, then the token
    bool rest = d.rest;
    u64 total = 0;
#pragma unroll 1
    for (int pass = rest ? 0 : 1; pass < 2; ++pass) {  // where p - q leaves nothing: p
        total = 0;
        for (int c = tid; c < a.pieces; c += kAT) total += __ldcg(&part[2 * c + pass]);
        total = block_scan(s_warp, total, &before);
        rest = pass == 0;
        if (total) break;
    }
    if (total == 0) {
        if (tid == 0) a.accept_len[r] = int32_t(n), a.next_tok[r] = -1;
        return;
    }
    const u64 target = scaled(fixed_u(a.u[r * a.T + drafts]), total);
    u64 base = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < a.pieces; c0 += kAT) {  // (a whole number of rounds: all threads take part)
        const int c = c0 + tid;
        const u64 here = c < a.pieces ? __ldcg(&part[2 * c + (rest ? 0 : 1)]) : 0ull;
        const u64 sum = block_scan(s_warp, here, &before);
        if (base + before <= target && target < base + before + here) s_piece = c, s_before = base + before;
        base += sum;
    }
    if (tid == 0) s_token = -1;
    __syncthreads();
    const int piece = s_piece;
    base = s_before;
    const int end = min((piece + 1) * a.each, V);
#pragma unroll 1
    for (int i0 = piece * a.each; i0 < end; i0 += kStep) {
        const int i = i0 + 4 * tid;
        const float4 x = read_x(i, end), y = read_y(i, end);
        u64 here = 0, stop = ~0ull;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {  // the sums, then the thread that holds the token
            at = pass ? -1 : 0;
            const u64 sum = quad(d, rest, i, x, y, whole, stop, &at);
            if (pass == 0) {
                here = sum;
                const u64 all = block_scan(s_warp, here, &before);
                before += base;
                base += all;
                if (target >= base) break;
                stop = before <= target && target < before + here ? target - before : ~0ull;
            } else if (stop != ~0ull) {
                s_token = at;
            }
        }
        if (target < base) break;
    }
    __syncthreads();
    if (tid == 0) a.accept_len[r] = int32_t(n), a.next_tok[r] = s_token;
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
