// kernels_attend_tc.cu -- attention over whole key tiles on the tensor cores
// (tcgen05), for parts with many query rows per key head: the prefix that
// all requests share, draft blocks.  The mathematics is kernels_attend.cu's;
// every key of these tiles is seen by every row, so there are no masks.
//
// A CTA has two slots, each a block of 128 query rows with its own region of
// tensor memory -- scores S (64 columns; the weights P take their place),
// output O (head_dim columns) and queries Q -- and its own four softmax
// warps (thread = row = tensor-memory lane) and issuing thread.  Units of
// 256 rows: slot s has rows 128 s .., both use every tile.  Units of 128
// rows: the slots take alternate tiles, and their results are added up by
// the join.  Per tile and slot:
//   S = Q K^T      4 or 8 products, A = Q from tensor memory, B = keys as
//                  they lie in the ring (K-major, 128-byte swizzle)
//   softmax        S to registers, maximum, exponentials, P back
//   O += P V       4 products, A = P from tensor memory, B = values as they
//                  lie in the ring (the channels contiguous)
// While one slot's warps work on S the tensor cores work for the other.  Q
// and P come from tensor memory so that shared memory only feeds B: a tile's
// keys and values are read once per slot, 256 cycles of 512 that the
// products take.  The issuing thread orders the products of its slot: S of
// tile i + 1 overwrites P of tile i after the product that reads it.
//
// O stays in tensor memory.  It is rescaled only when the maximum has grown
// by more than 2^8 since the last time (the exponentials are then at most
// 2^8, or, e4m3, 2^15 after the value's scale: inside fp16), by the slot's
// own warps, between two products.
//
// e4m3 tiles pass four converter warps, which write them as fp16 tiles in
// the same layout into a second ring.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "attend_device.cuh"
#include "device_common.cuh"
#include "tcgen05_common.cuh"

namespace w12 {

namespace {

constexpr float kNegInf = -INFINITY;
constexpr int kProdWarp = 8;   // copies
constexpr int kIssueWarp = 9;  // 9, 10: products of slot 0, 1
constexpr int kConvWarp = 12;  // 12 .. 15: e4m3 to fp16
constexpr uint32_t kTmem = 512, kSlotCols = 256, kOCol = 64, kQCol = 192;

template <int D, bool Q8, bool TWO>
struct TC {
    static constexpr int kThreads = Q8 ? 512 : 384;
    static constexpr int kOpTile = kAttTile * D * 2;    // keys or values of a tile as operands
    static constexpr int kOp = 2 * kOpTile;
    static constexpr int kIn = AttStage<D, Q8>::kBytes;
    static constexpr int kScales = (2 * kAttTile + 4) * 4;  // e4m3: per operand stage, scales and their bound
    static constexpr int kFixed = int(sizeof(AttShared)) + 1024 + (Q8 ? 8 * kScales : 0);
    // bf16: one ring, copies land as operands.  Units of 128 rows use stages
    // alternately by slot: an even number keeps a stage with one slot.
    static constexpr int SO = Q8 ? 4 : ((227 * 1024 - kFixed) / kOp > 8 ? 8 : ((227 * 1024 - kFixed) / kOp) & ~1);
    static constexpr int kInFit = (227 * 1024 - kFixed - SO * kOp) / kIn;
    static constexpr int SI = Q8 ? (kInFit > 8 ? 8 : kInFit) : SO;
    static constexpr int kRing = Q8 ? SI * kIn + SO * kOp : SO * kOp;
    static constexpr size_t kSmem = size_t(kRing) + kFixed;
    static_assert(SO >= 2 && SI >= 2 && kSmem <= 227 * 1024, "shared memory");
    static_assert((5 * 8 + 20) * 8 <= 1000, "barriers");
};

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// One 16-byte piece of an e4m3 row (16 channels) as two pieces of its fp16 row.
template <int D>
__device__ __forceinline__ void convert_piece(uint32_t src, uint32_t dst, int key, int c) {
    const uint4 x = lds128(D == 128 ? src + uint32_t(key * 128 + ((c ^ (key & 7)) << 4))
                                    : src + uint32_t(key * 64 + ((c ^ ((key >> 1) & 3)) << 4)));
    const uint32_t row = dst + uint32_t((c >> 2) * kAttTile * 128 + key * 128);
    const int p = 2 * (c & 3);
    sts128(row + uint32_t((p ^ (key & 7)) << 4), e4m3x2_lo_to_f16x2(x.x), e4m3x2_hi_to_f16x2(x.x),
           e4m3x2_lo_to_f16x2(x.y), e4m3x2_hi_to_f16x2(x.y));
    sts128(row + uint32_t(((p + 1) ^ (key & 7)) << 4), e4m3x2_lo_to_f16x2(x.z), e4m3x2_hi_to_f16x2(x.z),
           e4m3x2_lo_to_f16x2(x.w), e4m3x2_hi_to_f16x2(x.w));
}

template <int D, bool Q8, bool TWO>
__global__ void __launch_bounds__(Q8 ? 512 : 384, 1) attend_tc_kernel(const __grid_constant__ AttendArgs a) {
    using C = TC<D, Q8, TWO>;
    constexpr int SO = C::SO, SI = C::SI, KS = D / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    const uint32_t ops = base + uint32_t(Q8 ? SI * C::kIn : 0);  // the operand ring
    AttShared &sh = *reinterpret_cast<AttShared *>(smem + C::kRing);
    unsigned char *misc = smem + C::kRing + ((sizeof(AttShared) + 15) & ~size_t(15));
    uint64_t *in_full = reinterpret_cast<uint64_t *>(misc), *in_empty = in_full + SI;
    uint64_t *op_full = Q8 ? in_empty + SI : in_full, *op_empty = Q8 ? op_full + SO : in_empty;
    uint64_t *s_full = (Q8 ? op_empty + SO : in_empty + SI), *p_full = s_full + 2, *q_full = s_full + 4,
             *o_done = s_full + 6, *fin = s_full + 8;
    WaitCtl &ctl = *reinterpret_cast<WaitCtl *>(s_full + 10);
    uint32_t &s_tmem = *reinterpret_cast<uint32_t *>(reinterpret_cast<unsigned char *>(&ctl) + sizeof(WaitCtl));
    float *scales = reinterpret_cast<float *>(misc + 1008 - 16);  // [SO][2 * 64 + 4], 16-byte aligned
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (base & 1023u) {  // the swizzled boxes and operands need a 1024-byte aligned ring
        if (threadIdx.x == 0) record_error(a.err, W12_ERR_DEVICE);
        return;
    }
    if (threadIdx.x == 0) {
        constexpr uint32_t kUsers = TWO ? 2 : 1;  // issuing threads that use a stage
        for (int s = 0; s < SI; ++s) {
            mbar_init(&in_full[s], 1);
            mbar_init(&in_empty[s], Q8 ? 4 : kUsers);
        }
        if (Q8)
            for (int s = 0; s < SO; ++s) {
                mbar_init(&op_full[s], 4);
                mbar_init(&op_empty[s], kUsers);
            }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
            mbar_init(&q_full[s], 4);
            mbar_init(&o_done[s], 1);
            mbar_init(&fin[s], 1);
        }
        ctl.abort = 0;
        ctl.limit_ns = a.wait_ns ? a.wait_ns : kWaitLimitNs;
        mbar_fence_init();
    }
    if (warp == kIssueWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_launch_dependents();
    pdl_wait_previous();
    const AttPlan plan = att_plan(a, sh, C::kThreads);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = s_tmem;
    const AttendLine &ln = a.line[a.self];
    const int t0 = plan.t0, t1 = plan.t1;
    // the first of this slot's tiles from position k of a segment whose first
    // tile is the CTA's i0-th, and the step between them
    const auto first_tile = [](int i0, int slot) { return TWO ? 0 : (i0 & 1) != slot ? 1 : 0; };
    constexpr int kStep = TWO ? 1 : 2;

    if (warp == kProdWarp) {
        att_producer<D, Q8, SI>(a, plan, sh, base, in_full, in_empty, &ctl);
    } else if (warp == kIssueWarp || warp == kIssueWarp + 1) {
        // ------------------------------------------------------ products
        const int slot = warp - kIssueWarp;
        if (lane == 0) {
            const uint32_t ts = tmem + uint32_t(slot) * kSlotCols, to = ts + kOCol, tq = ts + kQCol;
            const uint32_t iqk = umma_idesc(Q8, kAttTile, false), ipv = umma_idesc(Q8, D, true);
            uint32_t n_seg = 0, n_p = 0;
            const auto scores = [&](int i) {
                const int s = i % SO;
                mbar_wait(&op_full[s], uint32_t(i / SO) & 1u, &ctl, a.err);
                tmem_fence_after();
                const uint64_t d = umma_desc_k(ops + uint32_t(s) * uint32_t(C::kOp));
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    umma_tmem_a(ts, tq + 8u * uint32_t(ks),
                                d + uint64_t(((ks >> 2) * kAttTile * 128 + 32 * (ks & 3)) >> 4), iqk, ks ? 1u : 0u);
                umma_arrive(&s_full[slot]);
            };
            for (int t = t0; t < t1;) {
                const AttSeg seg = att_locate(a, plan, sh, t);
                const int n = min(seg.left, t1 - t), i0 = t - t0, k0 = first_tile(i0, slot);
                t += n;
                if (k0 >= n) continue;
                mbar_wait(&q_full[slot], n_seg++ & 1u, &ctl, a.err);
                tmem_fence_after();
                scores(i0 + k0);
                for (int k = k0; k < n; k += kStep) {
                    const int i = i0 + k, s = i % SO;
                    mbar_wait(&p_full[slot], n_p++ & 1u, &ctl, a.err);
                    tmem_fence_after();
                    const uint64_t d = umma_desc_mn(ops + uint32_t(s) * uint32_t(C::kOp) + uint32_t(C::kOpTile),
                                                    kAttTile * 128);
#pragma unroll
                    for (int ks = 0; ks < kAttTile / 16; ++ks)
                        umma_tmem_a(to, ts + 8u * uint32_t(ks), d + uint64_t((ks * 2048) >> 4), ipv,
                                    (k > k0 || ks) ? 1u : 0u);
                    umma_arrive(&op_empty[s]);
                    if (k + kStep < n)
                        scores(i + kStep);
                    else
                        umma_arrive(&o_done[slot]);
                }
            }
            // every product issued has completed before the tensor memory is freed
            umma_arrive(&fin[slot]);
            mbar_drain(&fin[slot], 0u, ctl.limit_ns);
        }
        __syncwarp();
    } else if (Q8 && warp >= kConvWarp) {
        // ---------------------------------------------------- converters
        const int cw = warp - kConvWarp;
        // a quarter-warp's 8 lanes read the pieces 0-3 of an even key and 4-7
        // of the next (128 channels), then the others: neither the reads nor
        // the writes of the fp16 pieces share a bank
        const int odd = (lane >> 2) & 1;
        for (int t = t0; t < t1; ++t) {
            const int i = t - t0, si = i % SI, so = i % SO;
            mbar_wait(&in_full[si], uint32_t(i / SI) & 1u, &ctl, a.err);
            if (i >= SO) mbar_wait(&op_empty[so], uint32_t(i / SO - 1) & 1u, &ctl, a.err);
            const uint32_t src = base + uint32_t(si) * uint32_t(C::kIn);
            const uint32_t dst = ops + uint32_t(so) * uint32_t(C::kOp);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = 32 * h + 8 * cw + 2 * (lane >> 3) + odd;
#pragma unroll
                    for (int p = 0; p < D / 64; ++p)
                        convert_piece<D>(src + uint32_t(kv * AttStage<D, Q8>::kTile), dst + uint32_t(kv * C::kOpTile),
                                         key, (lane & 3) + (D == 128 ? 4 * (p ^ odd) : 0));
                }
            float *sc = scales + so * (2 * kAttTile + 4);
            const uint32_t ss = src + uint32_t(AttStage<D, Q8>::kScale);
            sc[32 * cw + lane] = __uint_as_float(lds32(ss + uint32_t(32 * cw + lane) * 4u));
            if (cw == 0) {  // the bound of the tile's value scales
                float top = fmaxf(__uint_as_float(lds32(ss + uint32_t(kAttTile + lane) * 4u)),
                                  __uint_as_float(lds32(ss + uint32_t(kAttTile + 32 + lane) * 4u)));
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                if (lane == 0) sc[2 * kAttTile] = exp_above(top) - 7.0f;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&op_full[so]);
                mbar_arrive(&in_empty[si]);
            }
        }
    } else if (warp < kProdWarp) {
        // ------------------------------------------------------- softmax
        const int slot = warp >> 2;
        const int row = 32 * (warp & 3) + lane;
        const uint32_t ts = tmem + uint32_t(slot) * kSlotCols + (uint32_t(32 * (warp & 3)) << 16);
        const uint32_t to = ts + kOCol, tq = ts + kQCol;
        uint32_t n_s = 0, n_seg = 0;
        for (int t = t0; t < t1;) {
            const AttSeg seg = att_locate(a, plan, sh, t);
            const int n = min(seg.left, t1 - t), i0 = t - t0, k0 = first_tile(i0, slot);
            t += n;
            const size_t entry = size_t(seg.unit + int(blockIdx.x)) * size_t(ln.halves) + (TWO ? 0 : slot);
            const int in_unit = (TWO ? 128 * slot : 0) + row;
            const bool valid = in_unit < seg.nrows;
            const bool warp_valid = __any_sync(0xFFFFFFFFu, valid);
            const size_t at = entry * size_t(ln.rt) + in_unit;
            if (k0 >= n) {  // no tile of the segment is this slot's
                if (valid) ln.part_ml[at] = make_float2(kNegInf, 0.0f);
                continue;
            }
            // ---- queries to tensor memory
            float sc = fabsf(a.scale_log2);
            if (warp_valid) {
                uint32_t q[D / 2];
#pragma unroll
                for (int j = 0; j < D / 2; ++j) q[j] = 0u;
                if (valid) {
                    const int rho = seg.row0 + in_unit, tok = rho / a.G, hq = seg.head * a.G + rho - tok * a.G;
                    const uint16_t *src = a.q + tok * a.q_stride + int64_t(hq) * D;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(src + 8 * j);
                        q[4 * j] = x.x, q[4 * j + 1] = x.y, q[4 * j + 2] = x.z, q[4 * j + 3] = x.w;
                    }
                }
                const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;  // scores grow with S
                if (Q8) {
                    uint32_t top = 0;
#pragma unroll
                    for (int j = 0; j < D / 2; ++j) top = max(top, max(q[j] & 0x7FFFu, (q[j] >> 16) & 0x7FFFu));
                    int e = int(top >> 7) - 127;
                    e = max(-100, min(126, e));
                    const float down = __uint_as_float(uint32_t(127 - e) << 23);
                    sc *= __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
                    for (int j = 0; j < D / 2; ++j)
                        q[j] = pack_f16(bf16_bits_to_float(q[j] & 0xFFFFu) * down, bf16_bits_to_float(q[j] >> 16) * down);
                }
#pragma unroll
                for (int j = 0; j < D / 2; ++j) q[j] ^= sign;
#pragma unroll
                for (int j = 0; j < D / 2; j += 32) tmem_store32(tq + uint32_t(j), q + j);
                tmem_wait_st();
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[slot]);

            float m = kNegInf, l = 0.0f;
            for (int k = k0; k < n; k += kStep) {
                const int i = i0 + k, so = i % SO;
                mbar_wait(&s_full[slot], n_s++ & 1u, &ctl, a.err);
                tmem_fence_after();
                if (warp_valid) {
                    float2 x[32];
                    tmem_load32(ts, reinterpret_cast<uint32_t *>(x));
                    tmem_load32(ts + 32u, reinterpret_cast<uint32_t *>(x + 16));
                    const float4 *tab = nullptr;
                    float lift = 0.0f;
                    if (Q8) {
                        // (the scores are there, so the tile is: this does not wait)
                        mbar_wait(&op_full[so], uint32_t(i / SO) & 1u, &ctl, a.err);
                        tab = reinterpret_cast<const float4 *>(scales + so * (2 * kAttTile + 4));
                        lift = scales[so * (2 * kAttTile + 4) + 2 * kAttTile];
                    }
                    tmem_wait_ld();
                    if (Q8) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float4 s4 = tab[j];
                            x[2 * j] = __fmul2_rn(x[2 * j], make_float2(s4.x, s4.y));
                            x[2 * j + 1] = __fmul2_rn(x[2 * j + 1], make_float2(s4.z, s4.w));
                        }
                    }
                    float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                    for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], fmaxf(x[j].x, x[j].y));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc + lift;
                    if (k == k0) {
                        m = top;
                    } else {
                        const bool grown = top - m > 8.0f;
                        if (__any_sync(0xFFFFFFFFu, grown)) {
                            const float f = grown ? ex2(m - top) : 1.0f;
                            if (grown) m = top;
                            l *= f;
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[32];
                                tmem_load32(to + uint32_t(c), o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_store32(to + uint32_t(c), o);
                            }
                            tmem_wait_st();
                        }
                    }
                    const float mu = m == kNegInf ? 0.0f : m;
                    const float2 sc2 = make_float2(sc, sc), mu2 = make_float2(-mu, -mu);
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    uint32_t p[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float2 e = __ffma2_rn(x[j], sc2, mu2);
                        e.x = ex2(e.x), e.y = ex2(e.y);
                        sum[j & 1] = __fadd2_rn(sum[j & 1], e);
                        if (Q8) {
                            const float2 v = reinterpret_cast<const float2 *>(tab)[kAttTile / 2 + j];
                            e = __fmul2_rn(e, v);
                        }
                        p[j] = Q8 ? pack_f16(e.x, e.y) : pack_bf16(e.x, e.y);
                    }
                    sum[0] = __fadd2_rn(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                    tmem_store32(ts, p);
                    tmem_wait_st();
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[slot]);
            }

            // ---- the segment's result
            mbar_wait(&o_done[slot], n_seg++ & 1u, &ctl, a.err);
            tmem_fence_after();
            if (warp_valid) {
                if (valid) ln.part_ml[at] = make_float2(m, l);
                float *dst = ln.part_o + at * D;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_load32(to + uint32_t(c), o);
                    tmem_wait_ld();
                    if (valid)
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<uint4 *>(dst + c + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kIssueWarp) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    }
}

// The dynamic shared-memory limit is raised once per device and variant.
template <int D, bool Q8, bool TWO>
int run(const AttendArgs &a, void *stream) {
    using C = TC<D, Q8, TWO>;
    static std::atomic<uint64_t> ready[4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return W12_ERR_CUDA;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(ready[dev >> 6].load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(attend_tc_kernel<D, Q8, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(C::kSmem)) != cudaSuccess)
            return W12_ERR_CUDA;
        ready[dev >> 6].fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_step(attend_tc_kernel<D, Q8, TWO>, a.line[a.self].grid, C::kThreads, C::kSmem, 1, stream, a);
}

}  // namespace

int launch_attend_tc(const AttendArgs &a, int dim, int kv, void *stream) {
    const bool q8 = kv == W12_KV_E4M3, two = a.line[a.self].rt == 256;
    if (dim == 128)
        return q8 ? (two ? run<128, true, true>(a, stream) : run<128, true, false>(a, stream))
                  : (two ? run<128, false, true>(a, stream) : run<128, false, false>(a, stream));
    return q8 ? (two ? run<64, true, true>(a, stream) : run<64, true, false>(a, stream))
              : (two ? run<64, false, true>(a, stream) : run<64, false, false>(a, stream));
}

}  // namespace w12
