// kernels_cut.cu -- what temperature, top-k, top-p and min-p leave of rows of
// logits: each row's largest logit, the lowest logit and index that stay, their whole
// weight and the drafted token's share of it (RowCut), by w12_sample's rules and with
// its whole-number weights (sample_device.cuh).  Nothing is drawn: the sampled
// verification needs single tokens' probabilities from most rows, and a draw from one
// per request.
//
// A row is read once: a cluster of CTAs holds it in shared memory, brought there by
// bulk copies.  The passes over it:
//  - the largest logit, as the pieces land;
//  - top-k (up to kCap / 2): with the largest logit the CTAs exchange the largest of
//    their warps' lanes' maxima, kT numbers a row; the k-th largest of these, found by
//    bisection, bounds the k-th largest logit from below.  What is not below it, little
//    more than k tokens, is gathered in the first CTA, which ranks it and cuts it by
//    top-p, too: no exponential of the others is needed;
//  - else the weights' sum, and for top-p a histogram of them: exact masses in 2048
//    bins, linear in (max - x) / t, over the tokens that can hold the boundary (one
//    lighter than (1 - top_p) 2^31 / V cannot: all such together weigh less than the
//    nucleus leaves out);
//  - the boundary: the first CTA finds the bin that holds it, its tokens are
//    gathered there and ranked, the other CTAs leave.  Where they are more than fit
//    (many equal logits), histograms over their composites come first.  Larger top-k:
//    the same with counts before the sum.
// What stays weighs what lies above the bin and what stays of its tokens, so no
// further pass over the row follows.
//
// What bounds it (rows of 151936): instructions and what waits between the cluster's
// barriers.  Without cuts 28 instructions a token (an exact exponential, its rounding, a
// 64-bit sum), 62 % of the issue slots: 240 fp32 rows 52 us, 21 for the bytes.  Top-p
// 59 a token, 55 %: 248 bf16 rows 120 us, of a CTA's 54 kcycles 19 for the sum and the
// bins (11 of them the two atomic additions a token), 8 for the gather, 6 for the
// ranking, the rest at barriers and in code that it has not met.  160 fp32 rows with
// top-k and 128 greedy ones 74 us.
// As few CTAs a row as hold it: with cuts in clusters of 16 instead of 4 or 8 top-p
// takes 164 us instead of 126, top-k 186 instead of 107 (with the draw).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "async_common.cuh"
#include "cluster_device.cuh"
#include "cut_device.cuh"
#include "draft_internal.h"
#include "sample_device.cuh"
#include "step_device.cuh"

namespace w12 {

namespace {

namespace cg = cooperative_groups;

constexpr int kT = 512, kPlainT = 256;  // threads per CTA, with cuts and without
constexpr int kW = kT / 32;
constexpr int kBins = 2048;
constexpr int kPieces = 2;          // bulk copies of a CTA's part of the row
constexpr int kMostCluster = 16;
constexpr int kCap = 680;           // tokens that are gathered
constexpr int kFew = 64;            // tokens that are ranked one against all
constexpr int kFine = 512;          // bins of the gathered tokens
constexpr float kSpan = 22.25f;     // e^-22.25 rounds to weight 0

// Which tokens a histogram is over: all (shift -1, bins linear in the exponent),
// or lo <= composite <= hi in bins of 2^shift composites.
struct Level {
    u64 lo, hi;
    int shift;
    int bin;       // the bin that is gathered; -1: nothing is cut
    float x0, x1;  // shift -1: its logits, and a little more
};

struct Small {
    uint64_t bar[kPieces];
    uint64_t fin;                  // (first CTA) the CTAs' last words have come
    WaitCtl ctl;
    float top[kMostCluster];
    u64 sums[2][kMostCluster];     // (first CTA) weights, those from floor_w on
    u64 ends[2][kMostCluster];     // (first CTA) largest and smallest composite of a bin
    u64 first[kMostCluster];
    float warp_top[kW];
    u64 warp_a[kW], warp_b[kW];
    Level level;
    u64 from;                      // the threshold so far
    uint32_t list_n;
    // the first CTA's search
    int bin;
    u64 above, lo, hi, thr, kept;
    uint32_t few_n;
};

// Behind it, for rows with cuts.  The bins are sums modulo 2^32 and sums of the upper
// 16-bit halves (with the 65536 logits a CTA can have, the lower halves' sums stay
// below 2^32, so the two give the whole), or counts; in the first CTA the cluster's
// sums take their place, as 64-bit numbers in two halves.
struct CutMem {
    uint32_t lo[kBins], hi[kBins];
    u64 list[kCap];
    uint32_t list_w[kCap];
    u64 few[kFew];
    uint32_t few_w[kFew];
    uint32_t fine_lo[kFine], fine_hi[kFine], fine_n[kFine];

    __device__ __forceinline__ float *tops() { return reinterpret_cast<float *>(fine_lo); }  // [kT], before those are used
};
static_assert(kFine >= kT, "the threads' maxima");
constexpr size_t kSmallBytes = (sizeof(Small) + 127) / 128 * 128, kCutBytes = (sizeof(CutMem) + 127) / 128 * 128;

// This CTA's part of a row in shared memory.
template <int DT>
struct Part {
    const unsigned char *x;
    int n;           // logits in it
    uint32_t first;  // index of its first
    bool inf;
    float mx, inv_t;

    __device__ __forceinline__ float clean(float v) const {
        if (inf) return v == INFINITY ? 0.0f : -INFINITY;
        return fmaxf(v, -INFINITY);
    }
    // logits i .. i + 3 (the part is padded to a multiple of 8 with -infinity)
    __device__ __forceinline__ void raw4(int i, float (&v)[4]) const {
        if (DT == W12_F32) {
            const float4 f = *reinterpret_cast<const float4 *>(x + 4 * i);
            v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
            const uint2 f = *reinterpret_cast<const uint2 *>(x + 2 * i);
            v[0] = bf16_bits_to_float(f.x & 0xFFFFu), v[1] = __uint_as_float(f.x & 0xFFFF0000u);
            v[2] = bf16_bits_to_float(f.y & 0xFFFFu), v[3] = __uint_as_float(f.y & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ float arg(float v) const { return __fmul_rn(__fsub_rn(v, mx), inv_t); }
    __device__ __forceinline__ uint32_t weight(float v) const { return __float2uint_rn(expf(arg(v)) * kOne31); }
    __device__ __forceinline__ u64 comp(float v, int i) const { return pack_key(v, first + uint32_t(i)); }
};

// The logit of a composite.
__device__ __forceinline__ float key_logit(u64 c) {
    const uint32_t k = uint32_t(c >> 32);
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// The larger of each half; a NaN loses against a number.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Adds v to the number AT bytes behind addr in shared memory where w >= least.
template <int AT>
__device__ __forceinline__ void add_if(uint32_t addr, uint32_t v, uint32_t w, uint32_t least) {
    asm volatile("{\n .reg .pred p;\n setp.ge.u32 p, %2, %3;\n @p red.shared.add.u32 [%0+%4], %1;\n}\n" ::"r"(addr), "r"(v), "r"(w),
                 "r"(least), "n"(AT)
                 : "memory");
}

// A block's sums of a and b (in warp 0's threads; the others keep their warp's).
template <int W>
__device__ __forceinline__ void block_sum2(Small &sh, u64 &a, u64 &b) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    a = warp_sum64(a), b = warp_sum64(b);
    if (lane == 0) sh.warp_a[warp] = a, sh.warp_b[warp] = b;
    __syncthreads();
    if (warp == 0) {
        a = warp_sum64(lane < W ? sh.warp_a[lane] : 0ull);
        b = warp_sum64(lane < W ? sh.warp_b[lane] : 0ull);
    }
}

// In one CTA: the bin in which the sum from bin 0 on, `above` before it, reaches
// `need`: sh.bin (-1: none), and what lies before it in sh.above.
template <int N, class M>
__device__ __forceinline__ void find(Small &sh, M mass, u64 above, u64 need) {
    constexpr int P = N / kT > 0 ? N / kT : 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    u64 m[P], sum = 0;
#pragma unroll
    for (int j = 0; j < P; ++j) {
        m[j] = tid * P + j < N ? mass(tid * P + j) : 0ull;
        sum += m[j];
    }
    const u64 incl = warp_scan64(sum, lane);
    __syncthreads();
    if (lane == 31) sh.warp_a[warp] = incl;
    if (tid == 0) sh.bin = -1;
    __syncthreads();
    // the warps before: lanes 0 .. 15 take one each
    const u64 w = warp_sum64(lane < warp ? sh.warp_a[lane & (kW - 1)] : 0ull);
    u64 before = above + w + incl - sum;
#pragma unroll
    for (int j = 0; j < P; ++j) {
        if (m[j] && before < need && need <= before + m[j]) sh.bin = tid * P + j, sh.above = before;
        before += m[j];
    }
    __syncthreads();
}

// The smallest shift that brings x below N (a power of two).
template <int N>
__device__ __forceinline__ int bits_above(u64 x) {
    return max(0, 64 - __clzll(static_cast<long long>(x)) - (31 - __clz(N)));
}

// In the first CTA: of its n gathered tokens, those from `from` on, the last one
// before which, together with `above`, less than `need` lies (by count or mass):
// sh.thr; sh.kept: with all before it.
__device__ __noinline__ void resolve(Small &sh, CutMem &cut, uint32_t n, u64 from, u64 above, u64 need, bool by_count) {
    const int tid = threadIdx.x, lane = tid & 31;
    __syncthreads();
    if (tid == 0) sh.lo = ~0ull, sh.hi = 0ull;
    __syncthreads();
    if (n > uint32_t(kFew)) {
        u64 hi = 0, lo = ~0ull;
        for (uint32_t i = tid; i < n; i += kT) {
            const u64 c = cut.list[i];
            if (c >= from) hi = umax64(hi, c), lo = lo < c ? lo : c;
        }
        hi = warp_max64(hi), lo = ~warp_max64(~lo);
        if (lane == 0) atomicMax(&sh.hi, hi), atomicMin(&sh.lo, lo);
    } else if (tid == 0) {
        sh.lo = from, sh.hi = ~0ull;
    }
    __syncthreads();
    u64 lo = sh.lo, hi = sh.hi;
    uint32_t left = n;
#pragma unroll 1
    while (left > uint32_t(kFew) && lo < hi) {
        const int shift = bits_above<kFine>(hi - lo);
        if (tid < kFine) cut.fine_lo[tid] = cut.fine_hi[tid] = cut.fine_n[tid] = 0u;
        __syncthreads();
        for (uint32_t i = tid; i < n; i += kT) {
            const u64 c = cut.list[i];
            if (c < lo || c > hi) continue;
            const int b = int((hi - c) >> shift);
            const uint32_t w = by_count ? 1u : cut.list_w[i];
            atomicAdd(&cut.fine_lo[b], w & 0xFFFFu);
            if (w >> 16) atomicAdd(&cut.fine_hi[b], w >> 16);
            atomicAdd(&cut.fine_n[b], 1u);
        }
        __syncthreads();
        find<kFine>(sh, [&](int b) { return u64(cut.fine_lo[b]) + (u64(cut.fine_hi[b]) << 16); }, above, need);
        const int b = sh.bin;
        if (b < 0) break;  // (not reached: the tokens hold it)
        above = sh.above;
        left = cut.fine_n[b];
        hi -= u64(b) << shift;
        const u64 width = (1ull << shift) - 1;
        lo = hi - lo > width ? hi - width : lo;
        __syncthreads();
    }
    if (tid == 0) sh.few_n = 0u, sh.thr = ~0ull;
    __syncthreads();
    for (uint32_t i = tid; i < n; i += kT)
        if (cut.list[i] >= lo && cut.list[i] <= hi) {
            const uint32_t at = atomicAdd(&sh.few_n, 1u);
            if (at < uint32_t(kFew)) cut.few[at] = cut.list[i], cut.few_w[at] = by_count ? 1u : cut.list_w[i];
        }
    __syncthreads();
    const uint32_t m = min(sh.few_n, uint32_t(kFew));
    int lanes = 2;  // per token
    while (lanes < 32 && m * 2 * lanes <= uint32_t(kT)) lanes *= 2;
    {
        const uint32_t i = tid / lanes, sub = tid & (lanes - 1);
        u64 before = 0;
        const u64 mine = i < m ? cut.few[i] : ~0ull;
        for (uint32_t j = sub; j < m; j += lanes)
            if (cut.few[j] > mine) before += cut.few_w[j];
        for (int o = 1; o < lanes; o <<= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
        if (i < m && sub == 0 && above + before < need) atomicMin(&sh.thr, mine);
        __syncthreads();
        if (i < m && sub == 0 && mine == sh.thr) sh.kept = above + before + cut.few_w[i];
    }
    __syncthreads();
}
static_assert(2 * kFew <= kT, "two threads a token");

// A CTA's last word to the first one: what this thread has written there before is
// seen after all_in.  The CTA may leave then.
__device__ __forceinline__ void hand_in(Small &sh) {
    asm volatile(
        "{\n .reg .b32 at;\n mapa.shared::cluster.u32 at, %0, 0;\n"
        " mbarrier.arrive.release.cluster.shared::cluster.b64 _, [at];\n}\n" ::"r"(smem_addr(&sh.fin))
        : "memory");
}
__device__ __forceinline__ void all_in(Small &sh, int *err) {
    mbar_wait(&sh.fin, 0u, &sh.ctl, err);
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

// CUTS: a top_k or top_p may be given.
template <int DT, bool CUTS>
__device__ __forceinline__ void cut_row(cg::cluster_group &cl, const CutArgs &a, const CutSide &s, int64_t r, unsigned char *smem) {
    constexpr int ES = DT == W12_F32 ? 4 : 2, kT = CUTS ? w12::kT : kPlainT, kW = kT / 32;
    Small &sh = *reinterpret_cast<Small *>(smem);
    CutMem &cut = *reinterpret_cast<CutMem *>(smem + kSmallBytes);
    unsigned char *buf = smem + kSmallBytes + (CUTS ? kCutBytes : 0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cs = int(cl.num_blocks()), me = int(cl.block_rank());

    Part<DT> row;
    const int64_t c0 = min(int64_t(me) * a.chunk, a.V);
    row.first = uint32_t(c0);
    row.n = int(min(a.V - c0, int64_t(a.chunk)));
    row.x = buf;
    const unsigned char *src = static_cast<const unsigned char *>(s.x) + (r * a.V + c0) * ES;
    const int64_t req = r / s.T;
    const int n8 = (row.n + 7) / 8 * 8;
    // (the request's numbers are on their way while the row is)
    const float t = s.temperature ? s.temperature[req] : 1.0f;
    uint32_t floor_w = 1;  // (above 2^31: no token stays)
    if (s.min_p) {
        const float m = s.min_p[req];
        if (m > 0.0f) floor_w = max(1u, min(0x80000001u, __float2uint_ru(fminf(m, 1.5f) * kOne31)));
    }
    const int32_t top_k = CUTS && s.top_k ? s.top_k[req] : 0;
    const bool by_k = CUTS && top_k > 0 && top_k < a.V;
    uint64_t p_fix = 1ull << 24;
    if (CUTS && s.top_p) {
        const float p = rintf(s.top_p[req] * 16777216.0f);
        if (p < 16777216.0f) p_fix = p > 0.0f ? uint64_t(p) : 0ull;  // (a NaN is no cut)
    }
    const bool by_p = CUTS && p_fix < (1ull << 24);
    int token = -1;  // the row's draft, for the first CTA
    float drafted = 0.0f;
    if (me == 0 && tid == 0 && r % s.T < s.drafts) {
        token = s.draft[req * s.drafts + r % s.T];
        if (token >= 0 && token < a.V) drafted = DT == W12_F32 ? static_cast<const float *>(s.x)[r * a.V + token]
                                                               : bf16_bits_to_float(static_cast<const uint16_t *>(s.x)[r * a.V + token]);
        if (token >= a.V) token = -1;
    }
    const auto put = [&](RowCut c, u64 total) {  // (one thread of the first CTA)
        c.inv = total ? __fdiv_rn(1.0f, __ull2float_rn(total)) : 0.0f;
        if (row.inf) c.mx = 3.402823466e38f, c.least = INFINITY;
        if (!total) c.least = INFINITY, c.last = -1;
        c.share = token >= 0 ? __fmul_rn(cut_weight(c, drafted, token).f, c.inv) : 0.0f;
        s.out[r] = c;
    };
    float best = -INFINITY;
    uint32_t best2 = 0xFF80FF80u;  // a pair of bf16 -infinities

    // ---- the row's part into shared memory, and its largest logit
    const auto top_of = [&](int i0, int i1) {  // multiples of 4
#pragma unroll 4
        for (int i = i0 + 4 * tid; i < i1; i += 4 * kT) {
            if constexpr (DT == W12_F32) {
                float v[4];
                row.raw4(i, v);
                best = fmaxf(best, fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
            } else {
                const uint2 f = *reinterpret_cast<const uint2 *>(row.x + 2 * i);
                best2 = max_bf16x2(best2, max_bf16x2(f.x, f.y));
            }
        }
    };
    const int piece = (n8 / kPieces + 7) / 8 * 8;
    if (s.vec) {
        if (tid == 0 && row.n > 0) {
            for (int q = 0; q < kPieces; ++q) {
                const int i0 = min(q * piece, row.n), i1 = q + 1 < kPieces ? min(i0 + piece, row.n) : row.n;
                mbar_expect_tx(&sh.bar[q], uint32_t((i1 - i0) * ES));
                if (i1 > i0)
                    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                     smem_addr(buf + i0 * ES)),
                                 "l"(src + i0 * ES), "r"(uint32_t((i1 - i0) * ES)), "r"(smem_addr(&sh.bar[q]))
                                 : "memory");
            }
        }
        // the part of the row that will take this one's place, into L2 (32 x 9 rows with
        // top-k 111 -> 107 us; without cuts five CTAs an SM do that for one another)
        if (CUTS && tid == 32) {
            int64_t q = r + (&s == &a.side[1] ? a.side[0].rows : 0) + a.ahead;
            const CutSide *o = &a.side[0];
            if (q >= o->rows) q -= o->rows, o = &a.side[1];
            if (q < o->rows && o->vec && row.n > 0)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const unsigned char *>(o->x) +
                                                                              (q * a.V + c0) * (o->f32 ? 4 : 2)),
                             "r"(uint32_t(row.n * (o->f32 ? 4 : 2)))
                             : "memory");
        }
        // what pads the part to eights (the copies end before it)
        if (tid < n8 - row.n) {
            if (DT == W12_F32)
                reinterpret_cast<float *>(buf)[row.n + tid] = -INFINITY;
            else
                reinterpret_cast<uint16_t *>(buf)[row.n + tid] = 0xFF80u;
        }
        if (row.n > 0)
            for (int q = 0; q < kPieces; ++q) {
                mbar_wait(&sh.bar[q], 0u, &sh.ctl, a.err);
                const int i0 = min(q * piece, row.n), i1 = q + 1 < kPieces ? min(i0 + piece, row.n) : row.n;
                top_of(i0, i1);  // (whole fours: 16 bytes hold them)
            }
        if (aborted(&sh.ctl) && tid == 0 && row.n > 0)  // let the copies in flight land
            for (int q = 0; q < kPieces; ++q) mbar_drain(&sh.bar[q], 0u, sh.ctl.limit_ns);
        if (DT != W12_F32) best = fmaxf(bf16_bits_to_float(best2 & 0xFFFFu), __uint_as_float(best2 & 0xFFFF0000u));
    } else {
#pragma unroll 8
        for (int i = tid; i < n8; i += kT) {
            if (DT == W12_F32) {
                const float v = i < row.n ? reinterpret_cast<const float *>(src)[i] : -INFINITY;
                reinterpret_cast<float *>(buf)[i] = v;
                best = fmaxf(best, v);
            } else {
                const uint16_t v = i < row.n ? reinterpret_cast<const uint16_t *>(src)[i] : uint16_t(0xFF80u);
                reinterpret_cast<uint16_t *>(buf)[i] = v;
                best = fmaxf(best, bf16_bits_to_float(v));
            }
        }
    }
    const bool quick = by_k && top_k <= kCap / 2 && t > 0.0f;
    float near_top = -INFINITY;  // quick: one of kT threads' maxima, the same in every CTA
    if (quick) {
        // ---- of each warp the largest 32 / cs of its threads' maxima, for all CTAs
        const int m = 32 / cs;
        uint32_t key = order_key(best), top = key;
        if (m < 32) {
#pragma unroll 1
            for (int j = 0; j < m; ++j) {
                const uint32_t k = __reduce_max_sync(0xFFFFFFFFu, key);
                if (lane == j) top = k;
                if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, key == k)) - 1) key = 0u;
            }
        }
        const float v = key_logit(u64(top) << 32);
        __syncthreads();
        cluster_started();
        if (lane < m)
            for (int c = 0; c < cs; ++c) cl.map_shared_rank(&cut, c)->tops()[(me * kW + warp) * m + lane] = v;
        cl.sync();
        near_top = cut.tops()[tid];
        const float w = key_logit(u64(__reduce_max_sync(0xFFFFFFFFu, order_key(near_top))) << 32);
        if (lane == 0) sh.warp_top[warp] = w;
        __syncthreads();
        float mx = w;
        for (int i = 0; i < kW; ++i) mx = fmaxf(mx, sh.warp_top[i]);
        row.inf = mx == INFINITY;
        row.mx = row.inf ? 0.0f : mx;
    } else {
        float m = best;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (lane == 0) sh.warp_top[warp] = m;
        __syncthreads();
        cluster_started();
        if (tid < cs) {
            for (int w = 0; w < kW; ++w) m = fmaxf(m, sh.warp_top[w]);
            cl.map_shared_rank(&sh, tid)->top[me] = m;
        }
        sync_sums();
        m = -INFINITY;
        for (int c = 0; c < cs; ++c) m = fmaxf(m, sh.top[c]);
        row.inf = m == INFINITY;
        row.mx = row.inf ? 0.0f : m;
    }
    if (row.mx == -INFINITY) {  // nothing can be sampled
        if (me == 0 && tid == 0) put(RowCut{0.0f, 1.0f, INFINITY, 1.0f, -1, -1}, 0ull);
        return;
    }
    if (!(t > 0.0f)) {  // the lowest index of the largest
        u64 first = 0;
        const float raw_mx = row.inf ? INFINITY : row.mx;
#pragma unroll 1
        for (int i = sh.top[me] == raw_mx ? 4 * tid : n8; i < n8; i += 4 * kT) {  // (most parts do not hold it)
            float v[4];
            row.raw4(i, v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (row.clean(v[j]) == row.mx && i + j < row.n) first = umax64(first, row.comp(row.mx, i + j));
        }
        u64 none = 0;
        first = warp_max64(first);
        if (lane == 0) sh.warp_a[warp] = first;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kW; ++w) first = umax64(first, sh.warp_a[w]);
            cl.map_shared_rank(&sh, 0)->first[me] = first;
            hand_in(sh);
        }
        if (me == 0 && tid == 0) {
            all_in(sh, a.err);
            for (int c = 0; c < cs; ++c) none = umax64(none, sh.first[c]);
            const int32_t one = int32_t(key_index(none));
            put(RowCut{row.mx, 1.0f, row.mx, 1.0f, one, one}, 1ull << 31);
        }
        return;
    }
    row.inv_t = fminf(__fdiv_rn(1.0f, t), 3.402823466e38f);
    const float unit = fmaxf(t, 2.9387359e-39f);  // logits per unit of the exponent
    Small *root = cl.map_shared_rank(&sh, 0);
    u64 thr = 0, kept = 0;  // (the first CTA's)
    uint32_t w_thr = 0;
    bool done = false;

    // ---- what the searches share
    constexpr float kMagic = 8388608.0f;  // an integer added to it is the low bits of the sum
    float slope = float(kBins - 1) / kSpan;
    const auto linear_bin = [&](float d) {
        return min(int(__float_as_uint(fmaf(d, -slope, kMagic)) - __float_as_uint(kMagic)), kBins - 1);
    };
    // The logits from x0 to x1: first marked, 64 at a time, then taken one by one (a
    // warp goes through f as often as one of its lanes has marks).
    const auto between = [&](float x0, float x1, auto f) {
#pragma unroll 1
        for (int q = 4 * tid; q < n8; q += 64 * kT) {
            u64 marks = 0;
#pragma unroll 2
            for (int k = 0; k < 16; ++k) {
                const int i = q + 4 * k * kT;
                if (i >= n8) break;
                float v[4];
                row.raw4(i, v);
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) m |= uint32_t(v[j] >= x0 && v[j] <= x1) << j;
                marks |= u64(m) << (4 * k);
            }
            for (; marks; marks &= marks - 1) {
                const int b = __ffsll(marks) - 1, i = q + 4 * (b >> 2) * kT + (b & 3);
                f(i, DT == W12_F32 ? reinterpret_cast<const float *>(buf)[i] : bf16_bits_to_float(reinterpret_cast<const uint16_t *>(buf)[i]));
            }
        }
    };
    const auto each = [&](auto f) {  // f(index, logit) of the part's logits, the padding too
#pragma unroll 2
        for (int i = 4 * tid; i < n8; i += 4 * kT) {
            float v[4];
            row.raw4(i, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) f(i + j, v[j]);
        }
    };
    // The cluster's bins in the first CTA, in the place of its own: every CTA adds up
    // its share.
    const auto add_up = [&]() {
        cl.sync();
        const int per = kBins / cs;
        CutMem *to = cl.map_shared_rank(&cut, 0);
        for (int b = me * per + tid; b < (me + 1) * per; b += kT) {
            u64 m = 0;
#pragma unroll 1
            for (int c0 = 0; c0 < cs; c0 += 4) {
                uint32_t lo[4], hi[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const CutMem *o = cl.map_shared_rank(&cut, min(c0 + c, cs - 1));
                    lo[c] = o->lo[b], hi[c] = o->hi[b];
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c0 + c < cs) m += u64(lo[c] - (hi[c] << 16)) + (u64(hi[c]) << 16);
            }
            to->lo[b] = uint32_t(m), to->hi[b] = uint32_t(m >> 32);
        }
        cl.sync();
    };
    const auto clear = [&]() {
        for (int i = tid; i < kBins; i += kT) cut.lo[i] = cut.hi[i] = 0u;
        __syncthreads();
    };
    const auto mass = [&](int b) { return u64(cut.lo[b]) | (u64(cut.hi[b]) << 32); };
    // One more token in the first CTA's list.
    const auto gather = [&](u64 c, uint32_t w) {
        const uint32_t at = atomicAdd(&root->list_n, 1u);
        if (at < uint32_t(kCap)) {
            CutMem *to = cl.map_shared_rank(&cut, 0);
            to->list[at] = c, to->list_w[at] = w;
        }
    };
    // The first CTA's word to all.
    const auto tell = [&](const Level &l) {
        if (tid == 0) {
            for (int c = 0; c < cs; ++c) {
                Small *o = cl.map_shared_rank(&sh, c);
                o->level = l, o->from = thr;
            }
        }
    };
    // The weight of the list's tokens from thr on.
    const auto listed = [&](uint32_t n, uint32_t least) {
        u64 mine = 0, none = 0;
        for (uint32_t i = tid; i < n; i += kT)
            if (cut.list[i] >= thr && cut.list_w[i] >= least) mine += cut.list_w[i];
        __syncthreads();
        block_sum2<kW>(sh, mine, none);
        if (tid == 0) sh.kept = mine;
        __syncthreads();
        return sh.kept;
    };
    // Finds the boundary: `need` by count or mass, of the bins that were added up.  The
    // tokens counted are those from `from` on with a weight of `light` at least.
    // After the last search (`last`) the other CTAs are not needed: false for them.
    const auto search = [&](u64 need, bool by_count, uint32_t light, bool last) {
        Level g{0ull, ~0ull, -1, 0, 0.0f, 0.0f};
        u64 above = 0;
#pragma unroll 1
        for (int depth = 0; depth < 8; ++depth) {
            if (me == 0) {
                find<kBins>(sh, mass, above, need);
                g.bin = sh.bin;
                if (g.bin >= 0) above = sh.above;
                if (g.shift < 0) {
                    // (a bin's end is half a step off the integer; 0.1 more, and the roundings)
                    const float d0 = g.bin == kBins - 1 ? -INFINITY : -(float(g.bin) + 0.6f) / slope, d1 = -(float(g.bin) - 0.6f) / slope;
                    const float pad = 1e-6f * fabsf(row.mx);
                    g.x0 = row.mx + d0 * unit * 1.000001f - pad, g.x1 = row.mx + d1 * unit * (d1 < 0.0f ? 0.999999f : 1.000001f) + pad;
                }
                tell(g);
                // (a cluster barrier lies behind the others' last look at it)
                if (tid == 0) sh.list_n = 0u;
            }
            cl.sync();
            g = sh.level;
            if (g.bin < 0) break;
            const u64 from = sh.from;
            u64 hi = 0, lo = ~0ull;
            const bool bounds = g.shift < 0 && !row.inf;
            between(bounds ? g.x0 : -INFINITY, bounds ? g.x1 : INFINITY, [&](int i, float v) {
                v = row.clean(v);
                const float d = row.arg(v);
                if (i >= row.n || (g.shift < 0 && (linear_bin(d) != g.bin || !(d > -kSpan)))) return;
                const u64 c = row.comp(v, i);
                if (c < from || (g.shift >= 0 && (c < g.lo || c > g.hi || int((g.hi - c) >> g.shift) != g.bin))) return;
                const uint32_t w = row.weight(v);
                if (w < light) return;
                hi = umax64(hi, c), lo = lo < c ? lo : c;
                gather(c, w);
            });
            cl.sync();
            const uint32_t n = root->list_n;
            if (n <= uint32_t(kCap)) {
                if (last && me != 0) return false;
                if (me == 0) {
                    resolve(sh, cut, n, thr, above, need, by_count);
                    if (sh.thr != ~0ull) thr = sh.thr, kept = sh.kept;  // (of masses)
                }
                break;
            }
            // too many: bins over their composites
            hi = warp_max64(hi), lo = ~warp_max64(~lo);
            if (lane == 0) sh.warp_a[warp] = hi, sh.warp_b[warp] = lo;
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w < kW; ++w) hi = umax64(hi, sh.warp_a[w]), lo = lo < sh.warp_b[w] ? lo : sh.warp_b[w];
                root->ends[0][me] = hi, root->ends[1][me] = lo;
            }
            cl.sync();
            if (me == 0) {
                g.hi = 0, g.lo = ~0ull;
                for (int c = 0; c < cs; ++c) g.hi = umax64(g.hi, sh.ends[0][c]), g.lo = g.lo < sh.ends[1][c] ? g.lo : sh.ends[1][c];
                g.shift = bits_above<kBins>(g.hi - g.lo);
                tell(g);
            }
            clear();
            cl.sync();
            g = sh.level;
            each([&](int i, float v) {
                v = row.clean(v);
                const u64 c = row.comp(v, i);
                if (i >= row.n || c < from || c < g.lo || c > g.hi) return;
                const uint32_t w = row.weight(v);
                if (w < light) return;
                const int b = int((g.hi - c) >> g.shift);
                atomicAdd(&cut.lo[b], by_count ? 1u : w);
                if (!by_count && w >> 16) atomicAdd(&cut.hi[b], w >> 16);
            });
            add_up();
        }
        if (me == 0) {
            w_thr = thr ? row.weight(key_logit(thr)) : 0u;
        }
        if (last) return me == 0;
        if (me == 0) tell(g);  // (the threshold)
        cl.sync();
        return true;
    };

    if (quick) {
        // ---- at least top_k tokens are among the maxima: the top_k-th of them bounds the
        // row's from below, to 22 / 2^14 of the exponent
        const float d = row.arg(row.clean(near_top));
        float end = -kSpan, above = 0.0f;  // (fewer of them than top_k have a weight: everything that has one)
        if (__syncthreads_count(d > -kSpan) >= top_k) {
#pragma unroll 1
            for (int i = 0; i < 14; ++i) {
                const float mid = 0.5f * (end + above);
                if (__syncthreads_count(d >= mid) >= top_k)
                    end = mid;
                else
                    above = mid;
            }
        }
        const float x0 = row.inf ? 0.0f : row.mx + end * unit * 1.000001f - 1e-6f * fabsf(row.mx);
        between(x0, INFINITY, [&](int i, float v) {
            v = row.clean(v);
            if (i >= row.n || !(row.arg(v) >= end)) return;
            const uint32_t w = row.weight(v);
            if (w) gather(row.comp(v, i), w);
        });
        cl.sync();
        const uint32_t n = root->list_n;
        done = n <= uint32_t(kCap);
        if (done) {
            if (me != 0) return;
            {
                u64 need = u64(top_k);
                bool by_count = true, cut_it = n > uint32_t(top_k) || end > -kSpan;  // (else: every token that has a weight)
#pragma unroll 1
                for (int stage = 0; stage < 2; ++stage) {
                    if (cut_it) {
                        resolve(sh, cut, n, thr, 0ull, need, by_count);
                        thr = sh.thr;
                    }
                    if (stage == 1 || !by_p) break;
                    kept = listed(n, 1u);
                    need = nucleus(p_fix, kept);
                    by_count = false, cut_it = need < kept;
                }
                kept = listed(n, floor_w);
            }
        }
    }
    const bool counted = CUTS && by_k && !done;
    if (!done) {
        uint32_t light = 1;  // lighter ones hold no boundary
        u64 heavy = 0;
#pragma unroll 1
        for (int stage = counted ? 0 : 1; stage < 2; ++stage) {
            u64 need = u64(top_k);
            if (CUTS && stage == 0) {
                // ---- the counts of all tokens that have a weight
                each([&](int i, float v) {
                    const float d = row.arg(row.clean(v));
                    if (i < row.n && d > -kSpan && row.weight(row.clean(v))) atomicAdd(&cut.lo[linear_bin(d)], 1u);
                });
                add_up();
            } else {
                // ---- the weights' sums, the bins of their masses
                const u64 from = counted ? sh.from : 0ull;
                if (CUTS && by_p && !counted) {
                    const uint32_t out = uint32_t((1u << 24) - uint32_t(p_fix)) << 7;  // (1 - p) 2^31
                    light = max(1u, __float2uint_rd(__fdividef(__uint2float_rz(out - 1u), float(a.V)) * 0.99999f));
                    slope = float(kBins - 1) / fminf(kSpan, __logf(__fdividef(kOne31, float(light))) + 0.02f);
                }
                u64 total = 0;
                if (!row.inf && from == 0 && floor_w <= 1) {
                    const uint32_t at = smem_addr(cut.lo), large = max(light, 65536u);
                    // (a NaN has weight 0 by itself)
                    const auto sum = [&](auto bins) {
                        constexpr int N = decltype(bins)::value ? 8 : 4;
#pragma unroll 1
                        for (int i = 4 * tid; i < n8; i += N * kT) {
                            float v[N];
                            uint32_t w[N], to[N];
#pragma unroll
                            for (int k = 0; k < N; k += 4) {
                                float(&q)[4] = *reinterpret_cast<float(*)[4]>(&v[k]);
                                if (k == 0 || i + k * kT < n8)
                                    row.raw4(i + k * kT, q);
                                else
                                    q[0] = q[1] = q[2] = q[3] = -INFINITY;
                            }
#pragma unroll
                            for (int j = 0; j < N; ++j) {
                                const float d = row.arg(v[j]);
                                w[j] = __float2uint_rn(expf(d) * kOne31);
                                if (decltype(bins)::value) {
                                    const uint32_t b = __float_as_uint(fminf(fmaf(d, -slope, kMagic), kMagic + float(kBins - 1)));
                                    to[j] = at + (b << 2) - (__float_as_uint(kMagic) << 2);
                                }
                            }
#pragma unroll
                            for (int j = 0; j < N; ++j) {
                                total = add_wide(total, w[j]);
                                if (decltype(bins)::value) {
                                    add_if<0>(to[j], w[j], w[j], light);
                                    add_if<4 * kBins>(to[j], w[j] >> 16, w[j], large);
                                }
                            }
                        }
                    };
                    if (CUTS && by_p)
                        sum(std::true_type());
                    else
                        sum(std::false_type());
                } else {
#pragma unroll 1
                    for (int i = tid; i < row.n; i += kT) {
                        const float v = row.clean(DT == W12_F32 ? reinterpret_cast<const float *>(buf)[i]
                                                                : bf16_bits_to_float(reinterpret_cast<const uint16_t *>(buf)[i]));
                        const uint32_t w = row.weight(v);
                        if (counted && row.comp(v, i) < from) continue;
                        total += w;
                        if (w >= floor_w) heavy += w;
                        if (CUTS && by_p && w >= light) {
                            atomicAdd(&cut.lo[linear_bin(row.arg(v))], w);
                            atomicAdd(&cut.hi[linear_bin(row.arg(v))], w >> 16);
                        }
                    }
                }
                block_sum2<kW>(sh, total, heavy);
                if (tid == 0) {
                    root->sums[0][me] = total, root->sums[1][me] = heavy;
                    if (!CUTS || !by_p) hand_in(sh);
                }
                if (CUTS && by_p)
                    add_up();
                else if (me == 0 && tid == 0)
                    all_in(sh, a.err);
                if (me == 0) {
                    kept = heavy = 0;
                    for (int c = 0; c < cs; ++c) kept += sh.sums[0][c], heavy += sh.sums[1][c];
                    need = nucleus(p_fix, kept);
                }
                if (!CUTS || !by_p) break;
            }
            if (!search(need, stage == 0, light, stage == 1)) return;
            if (stage == 0) clear();
        }
        // min_p above the threshold: all from floor_w on, else what the cuts left
        if (floor_w > 1u && floor_w > w_thr) kept = heavy;
    }
    if (me == 0 && tid == 0) {
        put(RowCut{row.mx, row.inv_t, thr ? key_logit(thr) : -INFINITY, float(floor_w), thr ? int32_t(key_index(thr)) : 0x7FFFFFFF, -1}, kept);
    }
}

template <bool CUTS>
__global__ void __launch_bounds__(CUTS ? kT : kPlainT, CUTS ? 2 : 5) cut_kernel(const __grid_constant__ CutArgs a) {
    cg::cluster_group cl = cg::this_cluster();
    extern __shared__ __align__(128) unsigned char smem[];
    Small &sh = *reinterpret_cast<Small *>(smem);
    constexpr int threads = CUTS ? kT : kPlainT;
    const int cs = int(cl.num_blocks());
    cluster_here();  // (its wait is behind the row's loads)
    if (threadIdx.x == 0) {
        for (int q = 0; q < kPieces; ++q) mbar_init(&sh.bar[q], 1);
        mbar_init(&sh.fin, cs);
        sh.ctl.abort = 0;
        sh.ctl.limit_ns = kWaitLimitNs;
        sh.list_n = 0u;
        mbar_fence_init();
    }
    if (CUTS) {
        uint32_t *h = reinterpret_cast<uint32_t *>(smem + kSmallBytes);
        for (int i = threadIdx.x; i < 2 * kBins; i += threads) h[i] = 0u;
    }
    pdl_launch_dependents();
    __syncthreads();
    pdl_wait_previous();
    int64_t r = int64_t(blockIdx.x) / cs;
    const int k = r >= a.side[0].rows;
    if (k) r -= a.side[0].rows;
    const CutSide &s = a.side[k];
    if (threadIdx.x == 0 && cl.block_rank() == 0 && k == 0 && r % s.T == 0) a.arrived[r / s.T] = 0u;
    if (s.f32)
        cut_row<W12_F32, CUTS>(cl, a, s, r, smem);
    else
        cut_row<W12_BF16, CUTS>(cl, a, s, r, smem);
    // The first CTA, whose shared memory the others read last, leaves after them (a
    // cluster barrier waits for the threads that have not left).
    if (cl.block_rank() == 0) sync_relaxed();
}

constexpr size_t kMostShared = 227 * 1024;
template <bool CUTS>
int run(const CutArgs &a, int cs, int es, void *stream) {
    static std::atomic<uint64_t> ready[4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return W12_ERR_CUDA;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(ready[dev >> 6].load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(cut_kernel<CUTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostShared)) != cudaSuccess ||
            cudaFuncSetAttribute(cut_kernel<CUTS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return W12_ERR_CUDA;
        ready[dev >> 6].fetch_or(bit, std::memory_order_relaxed);
    }
    const size_t smem = kSmallBytes + (CUTS ? kCutBytes : 0) + size_t(a.chunk) * es;
    return launch_step(cut_kernel<CUTS>, int((a.side[0].rows + a.side[1].rows) * cs), CUTS ? kT : kPlainT, smem, cs, stream, a);
}

}  // namespace

int launch_cut(CutArgs &a, void *stream) {
    const int es = a.side[0].f32 || (a.side[1].rows && a.side[1].f32) ? 4 : 2;
    const size_t over = kSmallBytes + (a.cuts ? kCutBytes : 0);
    const int64_t rows = a.side[0].rows + a.side[1].rows;
    // As few CTAs a row as five (with cuts: two, of twice the threads) fit on an SM, so
    // that some of them compute while others load or wait; more where there are few rows.
    // Without cuts, 240 rows of 151936 fp32 logits: 68 us in all (the draw then took 3
    // more) with 14 a row, 70 with 16 (whole clusters fill the GPU's parts worse); two an
    // SM of 256 threads 77, of 512 threads 75, four of 384 80.  (With cuts the CTAs share out powers of two.)
    // (304: two CTAs on each of 152 SMs.)
    const size_t most = (a.cuts ? 113 : 45) * 1024;
    const auto chunk = [&](int cs) { return ((a.V + cs - 1) / cs + 7) / 8 * 8; };
    int cs = 1;
    while (cs < kMostCluster && over + size_t(chunk(cs)) * es > most) cs += a.cuts ? cs : 1;
    while (cs < kMostCluster && chunk(cs) > 2048 && rows * cs * 2 <= 304) cs = cs * 2 < kMostCluster ? cs * 2 : kMostCluster;
    a.chunk = int32_t(chunk(cs));
    a.ahead = 304 / cs;
    static_assert(kSmallBytes + kCutBytes + (W12_SAMPLE_MAX_V / kMostCluster) * 4 <= kMostShared, "the largest row");
    static_assert(W12_SAMPLE_MAX_V / kMostCluster <= 65536, "16-bit halves of the weights");
    return a.cuts ? run<true>(a, cs, es, stream) : run<false>(a, cs, es, stream);
}

}  // namespace w12
