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
// A row is read once: a cluster of up to 8 CTAs keeps it in distributed
// shared memory (151936 fp32 logits: 74 KB a CTA).  Passes over the resident
// row: maximum (with the load); for top-k and top-p each a histogram of
// counts or weights over 2048 bins linear in (max - x) / t, merged over the
// cluster (each CTA adds up its share of the bins of all), then the one bin
// that holds the threshold is gathered and ranked in one CTA, after further
// histograms over its composite range while it is too full (many equal
// logits); last the weights by warp in index order, and the draw inside one
// warp's part.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>

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
constexpr int kCap = 1024;             // members of the threshold bin that are ranked directly
constexpr int kMaxCluster = 8;
constexpr float kOne31 = 2147483648.0f;
constexpr float kSpan = 22.25f;        // e^-22.25 rounds to weight 0

struct SampleShared {
    // counts; weights in two 16-bit halves (a bin's sums stay below 2^32 for
    // the 65536 logits a CTA can have at most)
    uint32_t cnt[kBins], lo[kBins], hi[kBins];
    u64 list[kCap];                             // composites of the threshold bin (CTA 0 of the cluster)
    uint32_t list_w[kCap];
    u64 slice[2][kMaxCluster];                  // per CTA of the cluster: what it sent (two buffers)
    u64 slice2[kMaxCluster];
    u64 warp_sum[kSW];
    u64 found_above;
    u64 thr;
    int found_bin;
    uint32_t list_n;
    int last;
};

__device__ __forceinline__ u64 umax64(u64 a, u64 b) { return a > b ? a : b; }

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

template <int DT>
struct Row {
    const void *x;  // this CTA's chunk (shared or global memory)
    int n;          // logits in it
    uint32_t first; // index of its first
    float mx, inv_t;

    __device__ __forceinline__ float at(int i) const {
        const float v = DT == W12_F32 ? static_cast<const float *>(x)[i]
                                      : bf16_bits_to_float(static_cast<const uint16_t *>(x)[i]);
        return v != v ? -INFINITY : v;  // NaN is never sampled
    }
    __device__ __forceinline__ u64 comp(float v, int i) const { return pack_key(v, first + uint32_t(i)); }
    // (max - x) / t as the exponent's argument, <= 0
    __device__ __forceinline__ float arg(float v) const { return __fmul_rn(v == mx ? 0.0f : __fsub_rn(v, mx), inv_t); }
    __device__ __forceinline__ uint32_t weight(float v) const {
        const float d = arg(v);
        if (!(d > -kSpan) || v == -INFINITY) return 0u;
        return __float2uint_rn(expf(d) * kOne31);
    }
};

// Which elements a histogram is over: composite >= thr, weight > 0, and, from
// the second level on, lo <= composite <= hi.
struct Range {
    u64 thr, lo, hi;
    int shift;   // bins of the composite range: (hi - composite) >> shift; -1: bins linear in the argument
    int bin;     // after a level: the bin that holds the threshold
};

__device__ __forceinline__ int arg_bin(float d) {
    const int b = int(-d * (float(kBins) / kSpan));
    return b < kBins ? b : kBins - 1;
}

template <int DT>
__device__ __forceinline__ bool in_bin(const Row<DT> &row, const Range &g, float v, u64 c) {
    if (c < g.thr) return false;
    if (g.shift < 0) return arg_bin(row.arg(v)) == g.bin;
    return c >= g.lo && c <= g.hi && int((g.hi - c) >> g.shift) == g.bin;
}

// The threshold composite of the tokens that are kept: by count (BYMASS
// false: the first `need`) or by weight (those before which less than
// ceil(p total) lies, at least one).  thr0: what an earlier cut has kept.
// Every thread of the cluster calls it and gets the result.
template <int DT, bool BYMASS>
__device__ u64 select(cg::cluster_group &cl, SampleShared &sh, const Row<DT> &row, u64 thr0, u64 need, uint64_t p_fix) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cs = int(cl.num_blocks()), me = int(cl.block_rank());
    Range g{thr0, 0ull, ~0ull, -1, 0};
    u64 above = 0;  // count or weight above the range
    for (int level = 0; level < 8; ++level) {
        for (int i = tid; i < kBins; i += kST) sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0u;
        __syncthreads();
        for (int i = tid; i < row.n; i += kST) {
            const float v = row.at(i);
            const u64 c = row.comp(v, i);
            if (c < thr0) continue;
            const uint32_t w = row.weight(v);
            if (w == 0u) continue;
            int b;
            if (g.shift < 0) {
                b = arg_bin(row.arg(v));
            } else {
                if (c < g.lo || c > g.hi) continue;
                b = int((g.hi - c) >> g.shift);
            }
            if (BYMASS) {
                atomicAdd(&sh.lo[b], w & 0xFFFFu);
                atomicAdd(&sh.hi[b], w >> 16);
            } else {
                atomicAdd(&sh.cnt[b], 1u);
            }
        }
        cl.sync();
        // this CTA's share of the bins, added up over the cluster; a thread
        // takes consecutive bins
        const int per = kBins / cs, pt = (per + kST - 1) / kST;  // bins per CTA and per thread (1 .. 4)
        u64 v[4], mine = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = 0;
            const int b = tid * pt + j;
            if (j < pt && b < per)
                for (int c = 0; c < cs; ++c) {
                    const SampleShared *o = cl.map_shared_rank(&sh, c);
                    v[j] += BYMASS ? u64(o->lo[me * per + b]) + (u64(o->hi[me * per + b]) << 16)
                                   : u64(o->cnt[me * per + b]);
                }
            mine += v[j];
        }
        u64 incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 z = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += z;
        }
        if (lane == 31) sh.warp_sum[warp] = incl;
        __syncthreads();
        u64 before = incl - mine, total = 0;
        for (int w = 0; w < kSW; ++w) {
            if (w < warp) before += sh.warp_sum[w];
            total += sh.warp_sum[w];
        }
        if (tid < cs) cl.map_shared_rank(&sh, tid)->slice2[me] = total;
        cl.sync();
        u64 all = 0;
        for (int c = 0; c < cs; ++c) {
            if (c < me) before += sh.slice2[c];
            all += sh.slice2[c];
        }
        if (level == 0) {
            if (BYMASS) {
                need = p_fix * (all >> 24) + ((p_fix * (all & 0xFFFFFFull) + 0xFFFFFFull) >> 24);
                need = need < 1 ? 1 : need;
            }
            if (need >= all) return thr0;  // nothing is cut (uniform over the cluster)
        }
        before += above;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (v[j] && before < need && need <= before + v[j]) {  // one thread of the cluster
                for (int c = 0; c < cs; ++c) {
                    SampleShared *o = cl.map_shared_rank(&sh, c);
                    o->found_bin = me * per + tid * pt + j;
                    o->found_above = before;
                }
            }
            before += v[j];
        }
        if (tid == 0 && me == 0) sh.list_n = 0u;
        cl.sync();
        g.bin = sh.found_bin;
        above = sh.found_above;
        // gather the bin's members in CTA 0
        SampleShared *root = cl.map_shared_rank(&sh, 0);
        u64 top = 0, bottom = ~0ull;
        for (int i = tid; i < row.n; i += kST) {
            const float x = row.at(i);
            const u64 c = row.comp(x, i);
            if (!in_bin(row, g, x, c)) continue;
            const uint32_t w = row.weight(x);
            if (w == 0u) continue;
            top = umax64(top, c);
            bottom = bottom < c ? bottom : c;
            const uint32_t at = atomicAdd(&root->list_n, 1u);
            if (at < kCap) {
                root->list[at] = c;
                root->list_w[at] = w;
            }
        }
        cl.sync();
        const uint32_t n = root->list_n;
        if (n <= kCap) {
            if (me == 0) {
                if (tid == 0) sh.thr = ~0ull;
                __syncthreads();
                for (uint32_t i = tid; i < n; i += kST) {
                    const u64 c = sh.list[i];
                    u64 b = above;
                    for (uint32_t j = 0; j < n; ++j)
                        if (sh.list[j] > c) b += BYMASS ? u64(sh.list_w[j]) : 1ull;
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

template <int DT>
__global__ void __launch_bounds__(kST) sample_kernel(const __grid_constant__ SampleArgs a) {
    cg::cluster_group cl = cg::this_cluster();
    extern __shared__ __align__(16) unsigned char smem[];
    SampleShared &sh = *reinterpret_cast<SampleShared *>(smem);
    unsigned char *buf = smem + ((sizeof(SampleShared) + 15) & ~size_t(15));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cs = int(cl.num_blocks()), me = int(cl.block_rank());
    const int64_t r = int64_t(blockIdx.x) / cs;
    constexpr int ES = DT == W12_F32 ? 4 : 2, VE = 16 / ES;
    pdl_launch_dependents();
    pdl_wait_previous();

    const int64_t c0 = int64_t(me) * a.chunk;
    Row<DT> row;
    row.first = uint32_t(c0 < a.V ? c0 : a.V);
    row.n = int(a.V - c0 > a.chunk ? a.chunk : a.V - c0 > 0 ? a.V - c0 : 0);
    const unsigned char *src = static_cast<const unsigned char *>(a.logits) + (r * a.V + row.first) * ES;
    row.x = a.resident ? static_cast<const void *>(buf) : static_cast<const void *>(src);
    row.mx = 0.0f, row.inv_t = 1.0f;

    // ---- load, maximum
    u64 best = 0;
    const int nv = a.vec ? row.n / VE : 0;
    for (int i0 = tid; i0 < nv; i0 += 4 * kST) {
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * kST < nv) x[k] = ldg_stream(src + size_t(i0 + k * kST) * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * kST;
            if (i >= nv) continue;
            if (a.resident) reinterpret_cast<uint4 *>(buf)[i] = x[k];
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (DT == W12_F32) {
                    const float v = __uint_as_float(w[q]);
                    if (v == v) best = umax64(best, row.comp(v, 4 * i + q));
                } else {
                    const float v0 = bf16_bits_to_float(w[q] & 0xFFFFu), v1 = bf16_bits_to_float(w[q] >> 16);
                    if (v0 == v0) best = umax64(best, row.comp(v0, 8 * i + 2 * q));
                    if (v1 == v1) best = umax64(best, row.comp(v1, 8 * i + 2 * q + 1));
                }
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
        if (v == v) best = umax64(best, row.comp(v, i));
    }
    best = warp_max64(best);
    if (lane == 0) sh.warp_sum[warp] = best;
    __syncthreads();
    if (tid < cs) {
        for (int w = 0; w < kSW; ++w) best = umax64(best, sh.warp_sum[w]);
        cl.map_shared_rank(&sh, tid)->slice[0][me] = best;
    }
    cl.sync();
    best = 0;
    for (int c = 0; c < cs; ++c) best = umax64(best, sh.slice[0][c]);
    {   // the logit back from its key
        const uint32_t k = uint32_t(best >> 32);
        row.mx = best ? __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k) : -INFINITY;
    }

    const int64_t req = r / a.T;
    const float t = a.temperature ? a.temperature[req] : 1.0f;
    int32_t token = -1;
    float prob = 0.0f;
    bool writer = me == 0 && tid == 0;
    if (row.mx == -INFINITY) {
        // nothing can be sampled
    } else if (!(t > 0.0f)) {
        token = int32_t(key_index(best));
        prob = 1.0f;
    } else {
        row.inv_t = __fdiv_rn(1.0f, t);
        u64 thr = 0;
        const int32_t k = a.top_k ? a.top_k[req] : 0;
        if (k > 0 && k < a.V) thr = select<DT, false>(cl, sh, row, thr, u64(k), 0ull);
        if (a.top_p) {
            const float p = rintf(a.top_p[req] * 16777216.0f);
            if (!(p >= 16777216.0f))
                thr = select<DT, true>(cl, sh, row, thr, 0ull, p > 0.0f ? uint64_t(p) : 0ull);
        }
        u64 floor_w = 1;
        if (a.min_p) {
            const float m = a.min_p[req];
            if (m > 0.0f) floor_w = umax64(1ull, u64(ceilf(fminf(m, 2.0f) * kOne31)));
        }
        // ---- weights by warp, in index order (each warp a contiguous part)
        const int part = ((row.n + kSW - 1) / kSW + 31) & ~31;
        const int p0 = min(warp * part, row.n), p1 = min(p0 + part, row.n);
        const auto kept = [&](int i) -> uint32_t {
            const float v = row.at(i);
            if (row.comp(v, i) < thr) return 0u;
            const uint32_t w = row.weight(v);
            return w >= floor_w ? w : 0u;
        };
        u64 sum = 0;
        for (int i = p0 + lane; i < p1; i += 32) sum += kept(i);
        sum = warp_sum64(sum);
        __syncthreads();
        if (lane == 0) sh.warp_sum[warp] = sum;
        __syncthreads();
        if (tid < cs) {
            u64 s = 0;
            for (int w = 0; w < kSW; ++w) s += sh.warp_sum[w];
            cl.map_shared_rank(&sh, tid)->slice[1][me] = s;
        }
        cl.sync();
        u64 before = 0, total = 0;
        for (int c = 0; c < cs; ++c) {
            if (c < me) before += sh.slice[1][c];
            total += sh.slice[1][c];
        }
        if (total > 0) {
            const float uf = a.u[r] * 16777216.0f;
            const uint64_t u = uf >= 16777215.0f ? 16777215ull : uf > 0.0f ? uint64_t(uf) : 0ull;
            const u64 target = (__umul64hi(u, total) << 40) | ((u * total) >> 24);
            for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
            writer = false;
            if (before <= target && target < before + sum) {  // one warp of the cluster
                for (int i0 = p0; i0 < p1; i0 += 32) {
                    const uint32_t w = i0 + lane < p1 ? kept(i0 + lane) : 0u;
                    u64 incl = w;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const u64 z = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                        if (lane >= o) incl += z;
                    }
                    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, before + incl > target);
                    if (hit) {
                        const int at = __ffs(hit) - 1;
                        if (lane == at) {
                            token = int32_t(row.first) + i0 + lane;
                            prob = __fdiv_rn(__uint2float_rn(w), __ull2float_rn(total));
                            writer = true;
                        }
                        break;
                    }
                    before += __shfl_sync(0xFFFFFFFFu, incl, 31);
                }
            }
        }
    }
    if (writer) {
        a.tokens[r] = token;
        if (a.prob) a.prob[r] = prob;
    }
    cl.sync();  // no CTA leaves while another may read its shared memory
    if (!a.accept_len || me != 0) return;
    // ---- the last row's cluster applies the acceptance rule
    if (tid == 0) {
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

constexpr size_t kSharedFixed = (sizeof(SampleShared) + 15) & ~size_t(15);
constexpr size_t kMostShared = 227 * 1024;

template <int DT>
int run(const SampleArgs &a, int cs, void *stream) {
    static std::atomic<uint64_t> ready[4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return W12_ERR_CUDA;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(ready[dev >> 6].load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(sample_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostShared)) !=
            cudaSuccess)
            return W12_ERR_CUDA;
        ready[dev >> 6].fetch_or(bit, std::memory_order_relaxed);
    }
    const size_t smem = kSharedFixed + (a.resident ? (size_t(a.chunk) * (DT == W12_F32 ? 4 : 2) + 15) / 16 * 16 : 0);
    return launch_step(sample_kernel<DT>, int(a.rows * cs), kST, smem, cs, stream, a);
}

}  // namespace

int launch_sample(SampleArgs &a, int dtype, int sms, void *stream) {
    (void)sms;
    const int es = dtype == W12_F32 ? 4 : 2;
    // Enough CTAs per row that each holds a few thousand logits, and the row
    // stays in shared memory.
    int cs = 1;
    while (cs < kMaxCluster && a.V > int64_t(cs) * 4096) cs *= 2;
    const int64_t chunk = ((a.V + cs - 1) / cs + 7) / 8 * 8;
    static_assert(W12_SAMPLE_MAX_V <= kMaxCluster * 65536, "16-bit halves of the weights");
    a.chunk = int32_t(chunk);
    a.resident = kSharedFixed + size_t(chunk) * es + 16 <= kMostShared;
    a.vec = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && (a.V * es) % 16 == 0;
    return dtype == W12_F32 ? run<W12_F32>(a, cs, stream) : run<W12_BF16>(a, cs, stream);
}

}  // namespace w12
