// kernels_sample.cu -- sampling with temperature, top-k, top-p and min-p from
// given random numbers, and the acceptance rule on the sampled tokens.
//
// Weights are fixed point: w_i = round(2^31 e^((x_i - max) / t)).  Their sums
// are whole numbers, so nucleus and draw do not depend on how a row is cut
// over threads and CTAs, and they are finer than an fp32 sum of
// probabilities (2^-32 of the largest weight each).  Tokens are ordered by
// logit, equal ones by index, lowest first: a token's composite key is
// (order-preserving key of the logit) << 32 | ~index, and what top-k and
// top-p keep is always "composite >= threshold".  A token of weight 0 (22 t
// below the largest logit) can neither be drawn nor change a sum.
//
// A row is read once: a cluster of 8 CTAs (16 where rows are few) keeps it in
// distributed shared memory (151936 fp32 logits: 74 KB a CTA).  The work on it:
//  - maximum, with the load;
//  - top_k up to 1024: the k-th largest of the threads' own maxima bounds the
//    k-th largest logit from below, so one histogram entry per thread gives a
//    bin (linear in (max - x) / t) above which all of the first k lie; they
//    are gathered in one CTA, which ranks them, cuts by top_p and min_p and
//    draws, alone;
//  - top_p over a whole row: the weights, kept in the logits' place (bf16:
//    beside them), and their sum; a sample of them -- the first sixteen of
//    every thread -- tells about where top_p of the sum is reached.  The tokens
//    around it, about 2000, are gathered in one CTA, which finds the boundary
//    from the exact sum of those above;
//  - where they are more than fit or do not hold it after all, and for larger
//    top_k: a histogram (64 bins per octave of weight) over the cluster of the
//    tokens that can matter -- a weight below (1 - top_p) of the mean cannot
//    hold the boundary -- the one bin that holds the boundary gathered and
//    ranked in one CTA, after further histograms over its composite range
//    while it is too full (many equal logits);
//  - the draw: a thread has consecutive tokens, so the sums of the threads
//    give the one that holds the token, and its warp looks at them again.
//
// What bounds it: the steps that wait for one another -- load, weights,
// counts, window, threshold, draw, each some 2000 cycles of work and a cluster
// barrier (16 rows of 151936, top-p: 30 us; one row, top-k: 10 us) -- and for
// many rows the instructions of the exact exponential and the 64-bit sums (128
// rows: 39 us for 78 MB).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>

#include "async_common.cuh"
#include "device_common.cuh"
#include "step_device.cuh"
#include "step_internal.h"

namespace w12 {

namespace {

namespace cg = cooperative_groups;

using u64 = unsigned long long;

constexpr int kST = 512;               // threads per CTA
constexpr int kSW = kST / 32;
constexpr int kBins = 2048;
constexpr int kCap = 1024;             // tokens that are ranked directly, one against all
constexpr int kWide = 2304;            // tokens that can be gathered for a nucleus' boundary
constexpr int kAround = 800;           // tokens to either side of where the sample sees the boundary
constexpr int kTaken = 16;             // sampled tokens per thread
constexpr int kMaxCluster = 16;        // (8 where rows are many)
constexpr float kOne31 = 2147483648.0f;
constexpr float kSpan = 22.25f;        // e^-22.25 rounds to weight 0

struct SampleSmall {
    u64 slice[2][kMaxCluster];         // per CTA of the cluster: what it sent
    u64 slice2[kMaxCluster];
    u64 warp_sum[kSW];
    u64 found_above;
    u64 thr;
    float top[kMaxCluster];
    float warp_top[kSW];
    int found_bin;
    uint32_t list_n;
    u64 lowest, highest;               // of the window's composites
    u64 mass;                          // what weighs more than the window
    uint32_t win_lo, win_end;          // window of weights
    int last;
};

// Only for top_k and top_p.  With 74 KB of logits just small enough for two
// CTAs on an SM, so that 16 rows of 8 CTAs run at once (36 clusters fit; with
// one CTA on an SM 15 would).
struct SampleCut {
    // counts and their sums over the cluster; or weights in two 16-bit halves
    // (a bin's sums stay below 2^32 for the 65536 logits a CTA can have)
    uint32_t lo[kBins], hi[kBins];
    union {                            // tokens that were gathered (CTA 0 of the cluster)
        struct {
            u64 list[kCap];            // their composites
            uint32_t list_w[kCap];     // and weights
        };
        u64 win[kWide];                // weight << 32 | index
    };
    union {
        uint32_t rank[kCap];
        uint16_t member[2 * kCap];     // of the window: the tokens of one bin
    };
};

constexpr size_t kSmallBytes = (sizeof(SampleSmall) + 15) & ~size_t(15), kCutBytes = (sizeof(SampleCut) + 15) & ~size_t(15);

// Where the weights are kept: fp32 logits are overwritten by theirs, bf16 ones
// (chunk: a multiple of 8) followed by them.
template <int DT>
__host__ __device__ constexpr size_t weights_at(int64_t chunk) {
    return DT == W12_F32 ? 0 : size_t(chunk) * 2;
}

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

__device__ __forceinline__ int arg_bin(float d) {
    const int b = int(-d * (float(kBins) / kSpan));
    return b < kBins ? b : kBins - 1;
}

// Bins of weights, largest first: 64 per octave of [1, 2^31].
__device__ __forceinline__ int weight_bin(uint32_t w) {
    return int(((158u << 23) - __float_as_uint(__uint2float_rz(w))) >> 17);
}
static_assert((31 << 6) < kBins, "octaves of weights");

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

// Which elements a histogram is over, from the second level on: lo <=
// composite <= hi, in bins of 2^shift composites; shift -1: bins of weights.
struct Range {
    u64 lo, hi;
    int shift;
    int bin;     // after a level: the bin that holds the boundary
};

// Adds up this CTA's share of the bins over the cluster (v: a thread's up to
// 4 bins from tid * pt on), and finds the boundary: the bin in which the sum
// from bin 0 on (`above` before it) reaches `need`.  Returns the whole sum.
// The bins may be written again when it returns.
template <bool BYMASS>
__device__ __forceinline__ void find_bin(cg::cluster_group &cl, SampleSmall &sh, SampleCut &cut, u64 above, u64 need,
                                         int *bin, u64 *before_bin) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cs = int(cl.num_blocks()), me = int(cl.block_rank());
    const int per = kBins / cs, pt = (per + kST - 1) / kST;  // bins per CTA and per thread (1 .. 4)
    cl.sync();
    u64 v[4], mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = 0;
        const int b = tid * pt + j;
        if (j < pt && b < per)
            for (int c = 0; c < cs; ++c) {
                const SampleCut *o = cl.map_shared_rank(&cut, c);
                v[j] += BYMASS ? u64(o->lo[me * per + b]) + (u64(o->hi[me * per + b]) << 16)
                               : u64(o->lo[me * per + b]);
            }
        mine += v[j];
    }
    const u64 incl = warp_scan64(mine, lane);
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    u64 before = incl - mine + above, total = 0;
    for (int w = 0; w < kSW; ++w) {
        if (w < warp) before += sh.warp_sum[w];
        total += sh.warp_sum[w];
    }
    if (tid < cs) cl.map_shared_rank(&sh, tid)->slice2[me] = total;
    if (tid == 0) sh.found_bin = -1;
    cl.sync();
    for (int c = 0; c < me; ++c) before += sh.slice2[c];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (v[j] && before < need && need <= before + v[j])  // one thread of the cluster
            for (int c = 0; c < cs; ++c) {
                SampleSmall *o = cl.map_shared_rank(&sh, c);
                o->found_bin = me * per + tid * pt + j;
                o->found_above = before;
            }
        before += v[j];
    }
    if (tid == 0 && me == 0) sh.list_n = 0u;
    cl.sync();
    *bin = sh.found_bin;
    *before_bin = sh.found_above;
}

// The cluster's counts (cut.lo added up) in every CTA's cut.hi; the caller's
// next write to cut.lo comes after another cluster barrier.
__device__ __forceinline__ void add_counts(cg::cluster_group &cl, SampleCut &cut) {
    const int cs = int(cl.num_blocks()), me = int(cl.block_rank()), g = kBins / 4 / cs;
    cl.sync();
    if (int(threadIdx.x) < g) {
        const int at = me * g + threadIdx.x;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        for (int c = 0; c < cs; ++c) {
            const uint4 x = reinterpret_cast<const uint4 *>(cl.map_shared_rank(&cut, c)->lo)[at];
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        for (int c = 0; c < cs; ++c) reinterpret_cast<uint4 *>(cl.map_shared_rank(&cut, c)->hi)[at] = v;
    }
    cl.sync();
}

// Calls put(place, i) for every logit i of the row's chunk that marks(i0)
// has a bit for (bit j: i0 + j), with places from the count in CTA 0 on, which
// a warp raises once for 64 logits a lane.
template <int DT, class M, class P>
__device__ __forceinline__ void collect(cg::cluster_group &cl, SampleSmall &sh, const Row<DT> &row, int each, M marks,
                                        P put) {
    const int lane = threadIdx.x & 31;
    uint32_t *count = &cl.map_shared_rank(&sh, 0)->list_n;
#pragma unroll 1
    for (int q0 = 0; q0 < each; q0 += 64) {
        u64 mask = 0;
        const int from = row.i0 + q0, to = min(row.i1, from + 64);
#pragma unroll 2
        for (int i = from; i < to; i += 4) mask |= u64(marks(i)) << (i - from);
        const uint32_t n = __popcll(mask);
        uint32_t at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t z = __shfl_up_sync(0xFFFFFFFFu, at, o);
            if (lane >= o) at += z;
        }
        uint32_t base = 0;
        if (lane == 31 && at) base = atomicAdd(count, at);
        at += __shfl_sync(0xFFFFFFFFu, base, 31) - n;
        for (; mask; mask &= mask - 1) put(at++, from + __ffsll(mask) - 1);
    }
}

__device__ __forceinline__ void gather(cg::cluster_group &cl, SampleSmall &sh, SampleCut &cut, u64 c, uint32_t w) {
    const uint32_t at = atomicAdd(&cl.map_shared_rank(&sh, 0)->list_n, 1u);
    if (at < uint32_t(kCap)) {
        SampleCut *root = cl.map_shared_rank(&cut, 0);
        root->list[at] = c;
        root->list_w[at] = w;
    }
}

// The threshold composite of the tokens that are kept: by count (BYMASS
// false: the first `need`) or by weight (those before which less than `need`
// lies), of those from thr0 on whose weight is at least w_min (the others
// cannot hold the boundary).  Every thread of the cluster calls it and gets
// the result.
template <int DT, bool BYMASS>
__device__ __noinline__ u64 select(cg::cluster_group &cl, SampleSmall &sh, SampleCut &cut, const Row<DT> &row_, u64 thr0,
                                   u64 need, uint32_t w_min) {
    const Row<DT> row = row_;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cs = int(cl.num_blocks()), me = int(cl.block_rank());
    Range g{0ull, ~0ull, -1, 0};
    u64 above = 0;  // count or weight above the range
    // calls f(composite, weight, bin) for the elements of the level
    const auto members = [&](auto f) {
#pragma unroll 1
        for (int i0 = row.i0; i0 < row.i1; i0 += 4) {
            uint32_t w[4];
            row.weight4(i0, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (w[j] < w_min || i0 + j >= row.i1) continue;
                const u64 c = thr0 || g.shift >= 0 ? row.comp(row.at(i0 + j), i0 + j) : ~0ull;
                if (c < thr0 || (g.shift >= 0 && (c < g.lo || c > g.hi))) continue;
                f(i0 + j, w[j], g.shift < 0 ? weight_bin(w[j]) : int((g.hi - c) >> g.shift));
            }
        }
    };
#pragma unroll 1
    for (int level = 0; level < 8; ++level) {
        for (int i = tid; i < kBins; i += kST) cut.lo[i] = cut.hi[i] = 0u;
        __syncthreads();
        members([&](int, uint32_t w, int b) {
            if (BYMASS) {
                atomicAdd(&cut.lo[b], w & 0xFFFFu);
                if (w >> 16) atomicAdd(&cut.hi[b], w >> 16);
            } else {
                atomicAdd(&cut.lo[b], 1u);
            }
        });
        find_bin<BYMASS>(cl, sh, cut, above, need, &g.bin, &above);
        if (g.bin < 0) return thr0;  // fewer than `need` of them: nothing is cut
        // gather the bin's members in CTA 0
        u64 top = 0, bottom = ~0ull;
        members([&](int i, uint32_t w, int b) {
            if (b != g.bin) return;
            const u64 c = row.comp(row.at(i), i);
            top = umax64(top, c);
            bottom = bottom < c ? bottom : c;
            gather(cl, sh, cut, c, w);
        });
        cl.sync();
        const uint32_t n = cl.map_shared_rank(&sh, 0)->list_n;
        if (n <= uint32_t(kCap)) {
            if (me == 0) {
                if (tid == 0) sh.thr = ~0ull;
                __syncthreads();
                for (uint32_t i = tid; i < n; i += kST) {
                    const u64 c = cut.list[i];
                    u64 b = above;
                    for (uint32_t j = 0; j < n; ++j)
                        if (cut.list[j] > c) b += BYMASS ? u64(cut.list_w[j]) : 1ull;
                    if (b < need) atomicMin(&sh.thr, c);
                }
                __syncthreads();
                if (tid < cs) cl.map_shared_rank(&sh, tid)->found_above = sh.thr;
            }
            cl.sync();
            return sh.found_above;
        }
        // too many: histogram over the members' composite range
        top = warp_max64(top);
        bottom = ~warp_max64(~bottom);
        if (lane == 0) sh.warp_sum[warp] = top;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kSW; ++w) top = umax64(top, sh.warp_sum[w]);
            for (int c = 0; c < cs; ++c) cl.map_shared_rank(&sh, c)->slice[0][me] = top;
        }
        __syncthreads();
        if (lane == 0) sh.warp_sum[warp] = bottom;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kSW; ++w) bottom = bottom < sh.warp_sum[w] ? bottom : sh.warp_sum[w];
            for (int c = 0; c < cs; ++c) cl.map_shared_rank(&sh, c)->slice[1][me] = bottom;
        }
        cl.sync();
        g.hi = 0, g.lo = ~0ull;
        for (int c = 0; c < cs; ++c) {
            g.hi = umax64(g.hi, sh.slice[0][c]);
            g.lo = g.lo < sh.slice[1][c] ? g.lo : sh.slice[1][c];
        }
        g.shift = 0;
        while (((g.hi - g.lo) >> g.shift) >= u64(kBins)) ++g.shift;
        cl.sync();  // the slices are read before the next level writes them
    }
    return thr0;  // not reached: a level divides the 64-bit range by 2048
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

// The cut and the draw among n <= kCap gathered tokens, by one CTA (all
// threads): the first k by rank, of those the nucleus p (2^24: all), of those
// the weights from floor_w on.
__device__ __forceinline__ void draw_from_list(SampleSmall &sh, SampleCut &cut, uint32_t n, uint32_t k, uint64_t p,
                                               uint32_t floor_w, uint64_t u, int32_t *token, float *prob, bool *writer) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // lanes per token (the whole CTA has work at any n), tokens at a time
    int lanes = 1;
    while (lanes < 32 && n * 2 * lanes <= uint32_t(kST)) lanes *= 2;
    const uint32_t sub = tid & (lanes - 1), team = tid / lanes, teams = kST / lanes;
    // a token's rank and the weight before it
    u64 before[2];
    uint32_t rank[2];
    u64 mine = 0;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint32_t i = team + q * teams;
        before[q] = 0, rank[q] = 0;
        if (i < n) {
            const u64 c = cut.list[i];
            for (uint32_t j = sub; j < n; j += lanes)
                if (cut.list[j] > c) {
                    before[q] += cut.list_w[j];
                    ++rank[q];
                }
        }
        for (int o = 1; o < lanes; o <<= 1) {
            before[q] += __shfl_xor_sync(0xFFFFFFFFu, before[q], o);
            rank[q] += __shfl_xor_sync(0xFFFFFFFFu, rank[q], o);
        }
        if (i < n && sub == 0 && rank[q] < k) mine += cut.list_w[i];
    }
    mine = warp_sum64(mine);
    __syncthreads();
    if (lane == 0) sh.warp_sum[warp] = mine;
    __syncthreads();
    u64 total = 0;
    for (int w = 0; w < kSW; ++w) total += sh.warp_sum[w];
    const u64 lim = p >= (1ull << 24) ? ~0ull : nucleus(p, total);
    // the weights that stay, in place of the others' zeros
    u64 kept = 0;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint32_t i = team + q * teams;
        if (i >= n || sub) continue;
        const uint32_t w = cut.list_w[i];
        cut.rank[i] = rank[q] < k && before[q] < lim && w >= floor_w ? w : 0u;
        kept += cut.rank[i];
    }
    kept = warp_sum64(kept);
    __syncthreads();
    if (lane == 0) sh.warp_sum[warp] = kept;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kSW; ++w) total += sh.warp_sum[w];
    if (total == 0) return;
    *writer = false;
    const u64 target = scaled(u, total);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint32_t i = team + q * teams;
        // the weight before it in index order (a composite's low half is ~index)
        u64 b = 0;
        if (i < n) {
            const uint32_t key = uint32_t(cut.list[i]);
            for (uint32_t j = sub; j < n; j += lanes)
                if (uint32_t(cut.list[j]) > key) b += cut.rank[j];
        }
        for (int o = 1; o < lanes; o <<= 1) b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        if (i >= n || sub) continue;
        if (b <= target && target < b + cut.rank[i]) {  // one thread
            *token = int32_t(key_index(cut.list[i]));
            *prob = __fdiv_rn(__uint2float_rn(cut.rank[i]), __ull2float_rn(total));
            *writer = true;
        }
    }
}

// The bin of cut.hi (counts) in which the sum from bin 0 on reaches `need`, -1:
// it does not.
__device__ __forceinline__ int find_count(SampleSmall &sh, const SampleCut &cut, uint32_t need) {
    static_assert(kBins == 4 * kST, "four bins a thread");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint4 v = reinterpret_cast<const uint4 *>(cut.hi)[tid];
    const uint32_t c[4] = {v.x, v.y, v.z, v.w}, mine = v.x + v.y + v.z + v.w;
    uint32_t before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t z = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += z;
    }
    if (lane == 31) sh.warp_sum[warp] = before;
    if (tid == 0) sh.found_bin = -1;
    __syncthreads();
    before -= mine;
    for (int w = 0; w < warp; ++w) before += uint32_t(sh.warp_sum[w]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (before < need && need <= before + c[j]) sh.found_bin = tid * 4 + j;
        before += c[j];
    }
    __syncthreads();
    return sh.found_bin;
}

// The smallest weight in the bins up to b (a bin's end is a float).
__device__ __forceinline__ uint32_t bin_end(int b) {
    return max(1u, __float2uint_ru(__uint_as_float((158u << 23) - (uint32_t(b + 1) << 17) + 1u)));
}

// From the sample's counts (cut.hi, by weight_bin) and what the nucleus leaves
// out: the window of weights, from bin_end to bin_end, around its boundary.
// `each`: logits per thread, of which kTaken were sampled.
__device__ __forceinline__ void set_window(SampleSmall &sh, const SampleCut &cut, u64 room, int each) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float part = each > kTaken ? float(kTaken) / float(each) : 1.0f;
    const float want = __ull2float_rn(room) * part;
    // the lightest first: the sums of what lies below are what counts
    const int b0 = kBins - 4 - 4 * tid;
    const uint4 v = *reinterpret_cast<const uint4 *>(&cut.hi[b0]);
    const uint32_t c[4] = {v.w, v.z, v.y, v.x};
    float w[4], mine = 0.0f;
    uint32_t mine_n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // (a bin's middle; the exact sum is taken later)
        w[j] = float(c[j]) * __uint_as_float((158u << 23) - (uint32_t(b0 + 3 - j) << 17) - (1u << 16));
        mine += w[j];
        mine_n += c[j];
    }
    float below = mine;
    uint32_t below_n = mine_n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_up_sync(0xFFFFFFFFu, below, o);
        const uint32_t z = __shfl_up_sync(0xFFFFFFFFu, below_n, o);
        if (lane >= o) below += x, below_n += z;
    }
    if (lane == 31) sh.warp_top[warp] = below, sh.warp_sum[warp] = below_n;
    if (tid == 0) sh.found_above = ~0ull;
    __syncthreads();
    float all = 0.0f;
    uint32_t all_n = 0;
    for (int q = 0; q < kSW; ++q) {
        if (q < warp) below += sh.warp_top[q], below_n += uint32_t(sh.warp_sum[q]);
        all += sh.warp_top[q], all_n += uint32_t(sh.warp_sum[q]);
    }
    below -= mine, below_n -= mine_n;
    {
        // sampled tokens below the boundary: all, where even they weigh less
        float x = below;
        uint32_t n = below_n;
        bool hit = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!hit && x + w[j] >= want) atomicMin(&sh.found_above, u64(n)), hit = true;
            x += w[j], n += c[j];
        }
    }
    __syncthreads();
    const uint32_t n = sh.found_above == ~0ull ? all_n : uint32_t(sh.found_above);
    // narrower, where the bins at its ends would make it too full (bf16: many
    // equal logits)
    for (int around = kAround; around >= kAround / 4; around /= 2) {
        const uint32_t d = uint32_t(float(around) * part) + 1u;
        const uint32_t from = n > d ? n - d : 0u, to = n + d;
        __syncthreads();
        if (tid == 0) sh.win_lo = 1u, sh.win_end = ~0u, sh.lowest = 0ull, sh.highest = all_n;
        __syncthreads();
        uint32_t at = below_n;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int b = b0 + 3 - j;
            if (c[j] && at <= from && from < at + c[j] && from > 0u) sh.win_lo = bin_end(b), sh.lowest = at;
            if (c[j] && at <= to && to < at + c[j]) sh.win_end = b > 0 ? bin_end(b - 1) : ~0u, sh.highest = at + c[j];
            at += c[j];
        }
        __syncthreads();
        if (float(sh.highest - sh.lowest) <= 0.85f * float(kWide) * part) break;
    }
}

// In one CTA: the bin of a histogram of weights (cut.lo, cut.hi) in which the
// sum, `above` before bin 0, reaches lim (-1: none); sh.found_above: before it.
__device__ __forceinline__ int boundary_bin(SampleSmall &sh, const SampleCut &cut, u64 above, u64 lim) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __syncthreads();
    if (tid == 0) sh.found_bin = -1;
    u64 v[4], mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = u64(cut.lo[tid * 4 + j]) + (u64(cut.hi[tid * 4 + j]) << 16);
        mine += v[j];
    }
    const u64 incl = warp_scan64(mine, lane);
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    u64 before = above + incl - mine;
    for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (v[j] && before < lim && lim <= before + v[j]) sh.found_bin = tid * 4 + j, sh.found_above = before;
        before += v[j];
    }
    __syncthreads();
    return sh.found_bin;
}

// In one CTA, with cut.lo and cut.hi all 0: the threshold composite among the n
// gathered tokens, which are those of the window: the last before which,
// together with the window's mass above, less than lim lies.  0: they do not
// hold it, or too many share its bin.  logit(index): of the row.
template <class L>
__device__ __forceinline__ u64 window_threshold(SampleSmall &sh, SampleCut &cut, uint32_t n, u64 lim, L logit) {
    const int tid = threadIdx.x, lane = tid & 31;
    // bins over the floats between the window's ends
    const uint32_t top = __float_as_uint(__uint2float_rz(min(sh.win_end, 0x80000000u)));
    const uint32_t span = top - __float_as_uint(__uint2float_rz(sh.win_lo));
    int shift = 0;
    while (span >> shift >= uint32_t(kBins)) ++shift;
    const auto bin_of = [&](uint32_t w) { return int((top - __float_as_uint(__uint2float_rz(w))) >> shift); };
    if (tid == 0) sh.list_n = 0u, sh.thr = ~0ull;
    for (uint32_t i = tid; i < n; i += kST) {
        const uint32_t w = uint32_t(cut.win[i] >> 32);
        const int b = bin_of(w);
        atomicAdd(&cut.lo[b], w & 0xFFFFu);
        if (w >> 16) atomicAdd(&cut.hi[b], w >> 16);
    }
    int bin = boundary_bin(sh, cut, sh.mass, lim);
    if (bin < 0) return 0;
    for (uint32_t i = tid; i < n; i += kST)
        if (bin_of(uint32_t(cut.win[i] >> 32)) == bin) {
            const uint32_t at = atomicAdd(&sh.list_n, 1u);
            if (at < 2u * kCap) cut.member[at] = uint16_t(i);
        }
    __syncthreads();
    uint32_t m = sh.list_n;
    if (m > 2u * kCap) return 0;
    // many of one weight: bins over their composites
#pragma unroll 1
    while (m > 128u) {
        __syncthreads();  // all have read the count that is reset below
        u64 c[4], top = 0, bottom = ~0ull;
        uint32_t id[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t i = tid + q * kST;
            if (i >= m) continue;
            id[q] = cut.member[i];
            const uint32_t x = uint32_t(cut.win[id[q]]);
            c[q] = pack_key(logit(x), x);
            top = umax64(top, c[q]);
            bottom = bottom < c[q] ? bottom : c[q];
        }
        const u64 above = sh.found_above;
        for (int i = tid; i < kBins; i += kST) cut.lo[i] = cut.hi[i] = 0u;
        if (tid == 0) sh.highest = 0ull, sh.lowest = ~0ull, sh.list_n = 0u;
        __syncthreads();
        top = warp_max64(top), bottom = ~warp_max64(~bottom);
        if (lane == 0) atomicMax(&sh.highest, top), atomicMin(&sh.lowest, bottom);
        __syncthreads();
        const u64 hi = sh.highest, width = hi - sh.lowest;
        int by = 0;
        while (width >> by >= u64(kBins)) ++by;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (tid + q * kST < m) {
                const uint32_t w = uint32_t(cut.win[id[q]] >> 32);
                const int b = int((hi - c[q]) >> by);
                atomicAdd(&cut.lo[b], w & 0xFFFFu);
                if (w >> 16) atomicAdd(&cut.hi[b], w >> 16);
            }
        bin = boundary_bin(sh, cut, above, lim);
        if (bin < 0) return 0;  // (not reached: the bin before held it)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (tid + q * kST < m && int((hi - c[q]) >> by) == bin) cut.member[atomicAdd(&sh.list_n, 1u)] = uint16_t(id[q]);
        __syncthreads();
        m = sh.list_n;
    }
    // the last ones against all
    u64 *comp = reinterpret_cast<u64 *>(cut.lo);  // (the bins are done with)
    __syncthreads();
    u64 mine = 0;
    if (tid < int(m)) {
        const uint32_t x = uint32_t(cut.win[cut.member[tid]]);
        comp[tid] = mine = pack_key(logit(x), x);
    }
    __syncthreads();
    if (tid < int(m)) {
        u64 b = sh.found_above;
        for (uint32_t j = 0; j < m; ++j)
            if (comp[j] > mine) b += cut.win[cut.member[j]] >> 32;
        if (b < lim) atomicMin(&sh.thr, mine);
    }
    __syncthreads();
    return sh.thr;
}

// CUT: top_k or top_p may be asked for.
template <int DT, bool CUT>
__global__ void __launch_bounds__(kST, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
    cg::cluster_group cl = cg::this_cluster();
    extern __shared__ __align__(16) unsigned char smem[];
    SampleSmall &sh = *reinterpret_cast<SampleSmall *>(smem);
    SampleCut &cut = *reinterpret_cast<SampleCut *>(smem + kSmallBytes);
    unsigned char *buf = smem + kSmallBytes + (CUT ? kCutBytes : 0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cs = int(cl.num_blocks()), me = int(cl.block_rank());
    const int64_t r = int64_t(blockIdx.x) / cs;
    constexpr int ES = DT == W12_F32 ? 4 : 2, VE = 16 / ES;
    cluster_here();  // (its wait is behind the row's loads)
    pdl_launch_dependents();
    pdl_wait_previous();

    const int64_t c0 = int64_t(me) * a.chunk;
    Row<DT> row;
    row.first = uint32_t(c0 < a.V ? c0 : a.V);
    row.n = int(a.V - c0 > a.chunk ? a.chunk : a.V - c0 > 0 ? a.V - c0 : 0);
    const unsigned char *src = static_cast<const unsigned char *>(a.logits) + (r * a.V + row.first) * ES;
    row.x = a.resident ? static_cast<const void *>(buf) : static_cast<const void *>(src);
    row.w = nullptr;
    row.vec = a.resident || a.vec;
    row.inf = false;
    row.mx = 0.0f, row.inv_t = 1.0f;
    // consecutive logits per thread, an odd number of fours: neither fp32 nor
    // bf16 fours of a warp share a bank (the same number in every CTA)
    const int each = (((a.chunk + kST - 1) / kST + 3) / 4 | 1) * 4;
    row.i0 = min(tid * each, row.n), row.i1 = min(row.i0 + each, row.n);
    const int64_t req = r / a.T;
    const float t = a.temperature ? a.temperature[req] : 1.0f;
    const int32_t top_k = CUT && a.top_k ? a.top_k[req] : 0;
    const bool few = CUT && top_k > 0 && top_k < a.V && top_k <= kCap && t > 0.0f;  // the first top_k in one CTA
    if (tid == 0) sh.last = 0;
    if (CUT)
        for (int i = tid; i < kBins; i += kST) cut.lo[i] = 0u;

    // ---- load, maximum (fmaxf drops a NaN)
    float best = -INFINITY;
    const int nv = a.vec ? row.n / VE : 0;
    for (int i0 = tid; i0 < nv; i0 += 8 * kST) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i0 + k * kST < nv) x[k] = ldg_stream(src + size_t(i0 + k * kST) * 16);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * kST;
            if (i >= nv) continue;
            if (a.resident) reinterpret_cast<uint4 *>(buf)[i] = x[k];
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (DT == W12_F32)
                    best = fmaxf(best, __uint_as_float(w[q]));
                else
                    best = fmaxf(best, fmaxf(bf16_bits_to_float(w[q] & 0xFFFFu), bf16_bits_to_float(w[q] >> 16)));
            }
        }
    }
    for (int i = nv * VE + tid; i < row.n; i += kST) {
        float v;
        if (DT == W12_F32) {
            v = reinterpret_cast<const float *>(src)[i];
            if (a.resident) reinterpret_cast<float *>(buf)[i] = v;
        } else {
            const uint16_t b = reinterpret_cast<const uint16_t *>(src)[i];
            if (a.resident) reinterpret_cast<uint16_t *>(buf)[i] = b;
            v = bf16_bits_to_float(b);
        }
        best = fmaxf(best, v);
    }
    {
        float m = best;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (lane == 0) sh.warp_top[warp] = m;
        __syncthreads();
        cluster_started();
        if (tid < cs) {
            for (int w = 0; w < kSW; ++w) m = fmaxf(m, sh.warp_top[w]);
            cl.map_shared_rank(&sh, tid)->top[me] = m;
        }
        sync_sums();
        m = -INFINITY;
        for (int c = 0; c < cs; ++c) m = fmaxf(m, sh.top[c]);
        row.inf = m == INFINITY;
        row.mx = row.inf ? 0.0f : m;
        best = row.clean(best);
    }

    int32_t token = -1;
    float prob = 0.0f;
    bool writer = me == 0 && tid == 0;
    uint32_t floor_w = 1;  // (above 2^31: no token stays)
    if (a.min_p) {
        const float m = a.min_p[req];
        if (m > 0.0f) floor_w = max(1u, min(0x80000001u, __float2uint_ru(fminf(m, 1.5f) * kOne31)));
    }
    uint64_t p_fix = 1ull << 24;
    if (CUT && a.top_p) {
        const float p = rintf(a.top_p[req] * 16777216.0f);
        if (p < 16777216.0f) p_fix = p > 0.0f ? uint64_t(p) : 0ull;  // (a NaN is no cut)
    }
    if (row.mx == -INFINITY) {
        // nothing can be sampled
    } else if (!(t > 0.0f)) {
        // the lowest index of the largest (a composite's low half is ~index)
        u64 first = 0;
#pragma unroll 1
        for (int i0 = row.i0; i0 < row.i1; i0 += 4) {
            float v[4];
            row.at4(i0, v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (v[j] == row.mx && i0 + j < row.i1) first = umax64(first, row.comp(v[j], i0 + j));
        }
        first = warp_max64(first);
        if (lane == 0) sh.warp_sum[warp] = first;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kSW; ++w) first = umax64(first, sh.warp_sum[w]);
            cl.map_shared_rank(&sh, 0)->slice[0][me] = first;
        }
        cl.sync();
        if (writer) {
            for (int c = 0; c < cs; ++c) first = umax64(first, sh.slice[0][c]);
            token = int32_t(key_index(first));
            prob = 1.0f;
        }
    } else {
        // finite for the smallest t, too: 0 (the largest logit's distance) times
        // infinity would be NaN
        row.inv_t = fminf(__fdiv_rn(1.0f, t), 3.402823466e38f);
        bool done = false;
        u64 thr = 0;
        if (CUT && few) {
            const float d = row.arg(best);
            if (d > -kSpan) atomicAdd(&cut.lo[arg_bin(d)], 1u);
            if (tid == 0) sh.list_n = 0u;
            add_counts(cl, cut);
            const int bin = find_count(sh, cut, uint32_t(top_k));
            // all logits down to the bin's end (fewer threads than top_k have
            // a weight: everything that has one)
            const float end = bin < 0 ? -kSpan : -(float(bin) + 1.01f) * (kSpan / float(kBins));
            SampleCut *root = cl.map_shared_rank(&cut, 0);
            collect(cl, sh, row, each, [&](int i) {
                float v[4];
                row.at4(i, v);
                uint32_t bits = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) bits |= uint32_t(row.arg(v[j]) >= end) << j;
                return bits;
            }, [&](uint32_t at, int i) {
                if (at >= uint32_t(kCap)) return;
                const float v = row.at(i);
                root->list[at] = row.comp(v, i);
                root->list_w[at] = row.weight(v);
            });
            cl.sync();
            const uint32_t n = cl.map_shared_rank(&sh, 0)->list_n;
            done = n <= uint32_t(kCap);
            if (done) {
                if (me == 0)
                    draw_from_list(sh, cut, n, uint32_t(top_k), p_fix, floor_w, fixed_u(a.u[r]), &token, &prob, &writer);
            } else {
                cl.sync();  // all have read the count
            }
        }
        if (!done) {
            // ---- weights, and their sums in index order
            uint32_t w_thr = 0;  // the threshold's weight
            const auto set_thr = [&](u64 c) {
                if (c == thr) return;
                thr = c;
                const uint32_t k = uint32_t(c >> 32);
                w_thr = row.weight(__uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k));
            };
            const auto kept = [&](int i, uint32_t w) -> uint32_t {
                if (CUT && (w < w_thr || (w == w_thr && w && thr && row.comp(row.at(i), i) < thr))) return 0u;
                return w >= floor_w ? w : 0u;
            };
            u64 mine = 0, before, total;  // this thread's sum, what lies before it
            const auto add_up = [&](int slot) {
                const u64 incl = warp_scan64(mine, lane);
                __syncthreads();
                if (lane == 31) sh.warp_sum[warp] = incl;
                __syncthreads();
                if (tid < cs) {
                    u64 s = 0;
                    for (int w = 0; w < kSW; ++w) s += sh.warp_sum[w];
                    cl.map_shared_rank(&sh, tid)->slice[slot][me] = s;
                }
                before = incl - mine;
                for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
                sync_sums();
                total = 0;
                for (int c = 0; c < cs; ++c) {
                    if (c < me) before += sh.slice[slot][c];
                    total += sh.slice[slot][c];
                }
            };
            const bool cuts = CUT && ((top_k > 0 && top_k < a.V) || p_fix < (1ull << 24));
            uint32_t *keep = cuts && a.keep_w ? reinterpret_cast<uint32_t *>(buf + weights_at<DT>(a.chunk)) : nullptr;
            const bool wide = cuts && !(top_k > 0 && top_k < a.V);  // top_p over the whole row
            if (CUT && wide && tid == 0) sh.list_n = 0u, sh.mass = 0;
            const auto take = [&](int i, const uint32_t (&w)[4]) {
                if (CUT && keep) reinterpret_cast<uint4 *>(keep)[i >> 2] = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) mine = add_wide(mine, (CUT && cuts) || w[j] >= floor_w ? w[j] : 0u);
                if (CUT && wide && i < row.i0 + kTaken)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (w[j]) atomicAdd(&cut.lo[weight_bin(w[j])], 1u);
            };
            int i = row.i0;
            if (a.resident && !row.inf) {  // whole fours in shared memory, without the general case's questions
                const uint32_t from = smem_addr(buf);
                const int full = row.i0 + (row.i1 - row.i0) / 4 * 4;
#pragma unroll 2
                for (; i < full; i += 4) {
                    float v[4];
                    if (DT == W12_F32) {
                        const uint4 f = lds128(from + uint32_t(i) * 4u);
                        v[0] = __uint_as_float(f.x), v[1] = __uint_as_float(f.y);
                        v[2] = __uint_as_float(f.z), v[3] = __uint_as_float(f.w);
                    } else {
                        const uint32_t x = lds32(from + uint32_t(i) * 2u), y = lds32(from + uint32_t(i) * 2u + 4u);
                        v[0] = bf16_bits_to_float(x & 0xFFFFu), v[1] = bf16_bits_to_float(x >> 16);
                        v[2] = bf16_bits_to_float(y & 0xFFFFu), v[3] = bf16_bits_to_float(y >> 16);
                    }
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = row.weight(fmaxf(v[j], -INFINITY));
                    take(i, w);
                }
            }
#pragma unroll 1
            for (; i < row.i1; i += 4) {
                uint32_t w[4];
                row.weight4(i, w);
                take(i, w);
            }
            if (keep) {
                row.w = keep;
                if (DT == W12_F32) row.x = src;  // (the few logits that are looked at again)
                __syncthreads();
            }
            add_up(0);
            if (CUT && wide) {
                const u64 lim = nucleus(p_fix, total);
                if (lim < total) {
                    add_counts(cl, cut);
                    set_window(sh, cut, total - lim, each);
                    const uint32_t lo = sh.win_lo, end = sh.win_end;
                    for (int i = tid; i < kBins; i += kST) cut.lo[i] = cut.hi[i] = 0u;
                    u64 more = 0;
                    SampleCut *root = cl.map_shared_rank(&cut, 0);
                    collect(cl, sh, row, each, [&](int i) {
                        uint32_t w[4], bits = 0;
                        row.weight4(i, w);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            more = add_wide(more, w[j] >= end ? w[j] : 0u);
                            bits |= uint32_t(w[j] - lo < end - lo) << j;
                        }
                        return bits;
                    }, [&](uint32_t at, int i) {
                        if (at < uint32_t(kWide)) root->win[at] = u64(row.weight_at(i)) << 32 | (row.first + uint32_t(i));
                    });
                    more = warp_sum64(more);
                    if (lane == 0 && more) atomicAdd(&cl.map_shared_rank(&sh, 0)->mass, more);
                    cl.sync();
                    if (me == 0) {
                        const uint32_t n = sh.list_n;
                        __syncthreads();
                        u64 c = 0;
                        if (n <= uint32_t(kWide))
                            c = window_threshold(sh, cut, n, lim, [&](uint32_t i) {
                                return row.clean(DT == W12_F32
                                                     ? static_cast<const float *>(a.logits)[r * a.V + i]
                                                     : bf16_bits_to_float(static_cast<const uint16_t *>(a.logits)[r * a.V + i]));
                            });
                        if (tid < cs) cl.map_shared_rank(&sh, tid)->slice2[0] = c;
                    }
                    cl.sync();
                    set_thr(sh.slice2[0]);
                }
            }
            if (CUT && cuts) {
                if (top_k > 0 && top_k < a.V) {
                    set_thr(select<DT, false>(cl, sh, cut, row, thr, u64(top_k), 1u));
                    mine = 0;
                    for (int i = row.i0; i < row.i1; ++i) {
                        const uint32_t w = row.weight_at(i);
                        if (w > w_thr || (w && w == w_thr && row.comp(row.at(i), i) >= thr)) mine += w;
                    }
                    add_up(1);
                }
                if (p_fix < (1ull << 24) && !(wide && thr)) {
                    const u64 lim = nucleus(p_fix, total);
                    // weights below it add up to at most total - lim
                    const u64 small = (total - lim) / u64(a.V);
                    if (lim < total)
                        set_thr(select<DT, true>(cl, sh, cut, row, thr, lim, uint32_t(small > 1 ? small : 1)));
                }
                mine = 0;
#pragma unroll 2
                for (int i = row.i0; i < row.i1; i += 4) {
                    uint32_t w[4];
                    row.weight4(i, w);
                    bool same = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        mine = add_wide(mine, w[j] > w_thr && w[j] >= floor_w ? w[j] : 0u);
                        same = same || w[j] == w_thr;
                    }
                    if (same)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (w[j] == w_thr) mine += kept(i + j, w[j]);
                }
                add_up(wide ? 1 : 0);  // (not the slot of the sum before it)
            }
            if (total > 0) {
                const u64 target = scaled(fixed_u(a.u[r]), total);
                writer = false;
                const uint32_t hit = __ballot_sync(0xFFFFFFFFu, before <= target && target < before + mine);
                if (hit) {  // one warp of the cluster: the thread's logits again, a lane each
                    const int src_lane = __ffs(hit) - 1;
                    u64 b = __shfl_sync(0xFFFFFFFFu, before, src_lane);
                    const int j1 = __shfl_sync(0xFFFFFFFFu, row.i1, src_lane);
                    for (int j0 = __shfl_sync(0xFFFFFFFFu, row.i0, src_lane); j0 < j1; j0 += 32) {
                        const uint32_t w = j0 + lane < j1 ? kept(j0 + lane, row.weight_at(j0 + lane)) : 0u;
                        const u64 incl = warp_scan64(u64(w), lane);
                        const uint32_t at = __ballot_sync(0xFFFFFFFFu, b + incl > target);
                        if (at) {
                            if (lane == __ffs(at) - 1) {
                                token = int32_t(row.first) + j0 + lane;
                                prob = __fdiv_rn(__uint2float_rn(w), __ull2float_rn(total));
                                writer = true;
                            }
                            break;
                        }
                        b += __shfl_sync(0xFFFFFFFFu, incl, 31);
                    }
                }
            }
        }
    }
    if (writer) {  // one thread of the cluster
        a.tokens[r] = token;
        if (a.prob) a.prob[r] = prob;
    }
    sync_relaxed();  // no CTA leaves while another may read its shared memory
    if (!a.accept_len) return;
    // ---- the CTA that has the last row's token applies the acceptance rule:
    // the thread that stored a token counts its row, as only it can order the
    // two (a release by the barrier above in its place: 16 rows 32.4 us, so 30.3)
    if (writer) {
        __threadfence();
        sh.last = atomicAdd(a.counter, 1u) == uint32_t(a.rows - 1);
    }
    __syncthreads();
    if (!sh.last) return;
    __threadfence();
    for (int64_t q = tid; q < a.R; q += kST) {
        int64_t n = a.T - 1;
        for (int64_t i = 0; i < a.T - 1; ++i)
            if (__ldcg(&a.draft[q * (a.T - 1) + i]) != __ldcg(&a.tokens[q * a.T + i])) {
                n = i;
                break;
            }
        a.accept_len[q] = int32_t(n);
        a.next_tok[q] = __ldcg(&a.tokens[q * a.T + n]);
    }
    if (tid == 0) *a.counter = 0u;
}

constexpr size_t kMostShared = 227 * 1024;
constexpr size_t kTwoShared = 113 * 1024;  // two CTAs on an SM

template <int DT, bool CUT>
int run_t(const SampleArgs &a, int cs, void *stream) {
    static std::atomic<uint64_t> ready[4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return W12_ERR_CUDA;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(ready[dev >> 6].load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(sample_kernel<DT, CUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostShared)) !=
                cudaSuccess ||
            cudaFuncSetAttribute(sample_kernel<DT, CUT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return W12_ERR_CUDA;
        ready[dev >> 6].fetch_or(bit, std::memory_order_relaxed);
    }
    const size_t smem = kSmallBytes + (CUT ? kCutBytes : 0) +
                        (a.keep_w ? weights_at<DT>(a.chunk) + size_t(a.chunk) * 4
                                  : a.resident ? (size_t(a.chunk) * (DT == W12_F32 ? 4 : 2) + 15) / 16 * 16 : 0);
    return launch_step(sample_kernel<DT, CUT>, int(a.rows * cs), kST, smem, cs, stream, a);
}

template <int DT>
int run(const SampleArgs &a, int cs, void *stream) {
    return a.top_k || a.top_p ? run_t<DT, true>(a, cs, stream) : run_t<DT, false>(a, cs, stream);
}

}  // namespace

int launch_sample(SampleArgs &a, int dtype, void *stream) {
    const int es = dtype == W12_F32 ? 4 : 2;
    // Enough CTAs per row that each holds a few thousand logits, and the row
    // stays in shared memory.  16 for up to 14 rows: so many such clusters run
    // at once (151936 logits, top-p: 8 rows 24 us with 16 CTAs, 30 with 8; 16
    // rows 41 and 31).
    int cs = 1;
    while (cs < (a.rows <= 14 ? kMaxCluster : 8) && a.V > int64_t(cs) * 4096) cs *= 2;
    const int64_t chunk = ((a.V + cs - 1) / cs + 7) / 8 * 8;
    static_assert(W12_SAMPLE_MAX_V <= 8 * 65536, "16-bit halves of the weights");
    a.chunk = int32_t(chunk);
    a.resident = kSmallBytes + kCutBytes + size_t(chunk) * es + 16 <= kMostShared;
    const size_t at = dtype == W12_F32 ? weights_at<W12_F32>(chunk) : weights_at<W12_BF16>(chunk);
    a.keep_w = (a.top_k || a.top_p) && kSmallBytes + kCutBytes + at + size_t(chunk) * 4 + 16 <= kTwoShared;
    a.vec = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && (a.V * es) % 16 == 0;
    return dtype == W12_F32 ? run<W12_F32>(a, cs, stream) : run<W12_BF16>(a, cs, stream);
}

}  // namespace w12
