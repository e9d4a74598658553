// kernels_fp4_tc.cu -- products with 4-bit weights for 17 .. 128 tokens, on
// tcgen05: the weights are expanded into tensor memory as operand A, the tokens
// (operand B) come from shared memory, the fp32 sums stay in tensor memory.
//
// Units of 256 columns x 128 k in one line over the CTAs, one CTA per SM (as in
// kernels_fp4.cu).  A unit is two tiles of 128 columns that share its tokens: at
// 128 tokens a unit's tokens are 32 KB beside 18 KB of weights, and one tile alone
// would read them twice.  Roles:
//  - 16 warps expand, in two groups that take the units in turn (so that one group's
//    waits lie under the other's work): thread (w, l) of a group has row 32 (w % 4) + l
//    of both tiles and half h = w / 4 of the 128 k, 64 weights of each, expanded in
//    registers and stored with tcgen05.st into the tile's A buffer of that group
//    (column j: k = 2 j, 2 j + 1);
//  - one warp copies the weights (one bulk copy a unit), one the tokens (two boxes of
//    64 k x MP tokens, 128-byte swizzle);
//  - two warps issue, one per tile: 8 UMMAs a unit (M = 128, N = MP, K = 16) into the
//    tile's sums, committed to the A buffer's and the token slot's barriers;
//  - at the end of a part of a tile's piece the group adds its sums up, at the end of the
//    piece it writes y, or the piece's place for the fix-up.
// What bounds it: at 128 tokens the UMMAs (64 cycles each, 1024 a unit) and the
// expansion (some 2900 warp-instructions a unit, 725 cycles of the four schedulers)
// beside one another, where the weight stream would take 815; tensor pipe 47 %, issue
// 51 %.  At fewer tokens a unit takes some 1500 cycles, twice what the expansion issues:
// its warps wait for one of two A buffers a tile.  5120 x 34816 at 32 / 64 / 128 tokens:
// 32.2 / 32.9 / 37.0 us (14.8 for the bytes, 23.5 for 128 tokens' products at the rate of a
// large matrix product).
// The tensor core cuts where it adds, so a sum of one sign drifts with its length.  After
// kSpan units a part's sums are taken out of tensor memory and added up in fp32, in the
// piece's place for the fix-up.  Sums of one sign, low by at most (of themselves): K = 5120
// 4e-6, any longer K 7e-6 (kept in tensor memory throughout: 2.5e-5 at 17408, 5e-4 at
// 131072, rising), where a rounding to bf16 is up to 4e-3; signs that differ: 2e-6 of y's
// norm.  Spans of 32 / 16 units: 2e-6 / 6e-7, but a part's end lets the tensor core wait:
// 5120 x 34816 at 32 / 128 tokens 33.8 / 42.5 and 35.3 / 47.3 us instead of 32.2 / 37.0.
//
// Every wait is bounded; after a timeout every role runs to its end without waiting,
// the producers let their copies land, and the issuers wait for their UMMAs and for the
// other warps' last use of the tensor memory before it is freed.
#include <cuda.h>
#include <cuda_runtime.h>

#include "draft_internal.h"
#include "fp4_device.cuh"
#include "step_device.cuh"
#include "stream_device.cuh"
#include "tcgen05_common.cuh"

namespace w12 {

namespace {

constexpr int kDW = 16;            // warps that expand
constexpr int kDT = kDW * 32;
constexpr int kWeightWarp = kDW, kTokenWarp = kDW + 1, kIssueWarp = kDW + 2;  // two issuers
constexpr int kThreads = (kDW + 4) * 32;
constexpr uint32_t kTmemCols = 512;
constexpr int kSpan = 64;  // units of a part (8192 k)

template <int MP>
struct TCfg {
    static constexpr int kX = MP * 256;                  // a unit's tokens: two boxes of MP rows x 128 bytes
    static constexpr int SX = 3;
    static constexpr int kBars = 1024;
    static constexpr int kFit = (227 * 1024 - kBars - SX * kX) / kFp4Unit;
    static constexpr int SW = kFit > 8 ? 8 : kFit / 2 * 2;  // even: a stage's units are one group's
    static constexpr int kBarOff = SX * kX + SW * kFp4Unit;
    static constexpr size_t kSmem = size_t(kBarOff) + kBars;
    // sums of tile t at columns t MP, its A buffer a at kA + (2 t + a) 64
    static constexpr uint32_t kA = 2 * MP < 64 ? 64u : uint32_t(2 * MP);
    static_assert(kA + 4 * 64 <= kTmemCols, "tensor memory");
    static_assert(SW >= 3, "ring");
};

struct Bars {
    uint64_t full_w[8], empty_w[8];  // the unit's weights; its group's 8 warps have read them
    uint64_t full_x[3], empty_x[3];  // its tokens; both tiles' UMMAs have read them
    uint64_t a_full[2][2], a_empty[2][2];  // [tile][buffer]: expanded (8 warps); read by the UMMAs
    uint64_t sum_full[2], sum_empty[2];    // a piece's sums; read (8 warps)
    uint64_t fin[2];
    uint64_t out;                          // the warps that expand (16) have read their last sums
    uint32_t tmem;
    int last;
    WaitCtl ctl;
};

__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// After the wait: the loaded registers are used from here on.
__device__ __forceinline__ void tmem_landed16(uint32_t (&r)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]),
                     "+r"(r[i + 7]));
}

// *p += v, in L2 (no other thread's number: the order of a thread's additions is its own),
// and the number back.
__device__ __forceinline__ void add_to(float *p, float v) {
    asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
}
__device__ __forceinline__ float load_back(const float *p) {
    float v;
    asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

template <int MP>
__global__ void __launch_bounds__(kThreads, 1) fp4_tc_kernel(const __grid_constant__ Fp4Batch b) {
    using C = TCfg<MP>;
    constexpr int SW = C::SW, SX = C::SX;
    extern __shared__ __align__(1024) unsigned char smem[];
    if (smem_addr(smem) & 1023u) {  // the boxes and descriptors need it; reported, not used
        if (threadIdx.x == 0) record_error(b.err, W12_ERR_DEVICE);
        return;
    }
    Bars &bar = *reinterpret_cast<Bars *>(smem + C::kBarOff);
    static_assert(sizeof(Bars) <= C::kBars, "barriers");
    const uint32_t xbase = smem_addr(smem), wbase = xbase + uint32_t(SX * C::kX);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int u0, u1;
    fp4_units(b, u0, u1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < SW; ++s) mbar_init(&bar.full_w[s], 1), mbar_init(&bar.empty_w[s], kDW / 2);
        for (int s = 0; s < SX; ++s) mbar_init(&bar.full_x[s], 1), mbar_init(&bar.empty_x[s], 2);
        for (int t = 0; t < 2; ++t) {
            for (int a = 0; a < 2; ++a) mbar_init(&bar.a_full[t][a], kDW / 2), mbar_init(&bar.a_empty[t][a], 1);
            mbar_init(&bar.sum_full[t], 1);
            mbar_init(&bar.sum_empty[t], kDW / 2);
            mbar_init(&bar.fin[t], 1);
        }
        mbar_init(&bar.out, kDW);
        bar.ctl.abort = 0;
        bar.ctl.limit_ns = kWaitLimitNs;
        mbar_fence_init();
    }
    if (warp == kIssueWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bar.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = bar.tmem;
    WaitCtl *ctl = &bar.ctl;
    if (threadIdx.x == 0) pdl_launch();

    if (warp == kWeightWarp) {
        if (lane != 0 || u0 >= u1) return;
        if (!b.early_weights) pdl_wait();
        const uint64_t pol = l2_evict_first_policy();
        SCur c = s_at(b, u0);
        int i = 0;
        for (int u = u0; u < u1; ++u, ++i) {
            const int s = i % SW;
            if (i >= SW && (!mbar_wait(&bar.empty_w[s], uint32_t(i / SW - 1) & 1u, ctl, b.err) || aborted(ctl))) break;
            const Fp4One &g = b.g[c.gi];
            mbar_expect_tx(&bar.full_w[s], kFp4Unit);
            bulk_copy(wbase + uint32_t(s) * kFp4Unit, g.units + (size_t(c.nb) * g.KG + c.kg) * kFp4Unit, kFp4Unit, &bar.full_w[s], pol);
            s_next(b, c);
        }
        if (aborted(ctl))  // let the copies in flight land
            for (int k = i > SW ? i - SW : 0; k < i; ++k) mbar_drain(&bar.full_w[k % SW], uint32_t(k / SW) & 1u, ctl->limit_ns);
        return;
    }
    pdl_wait();
    if (warp == kTokenWarp) {
        if (lane != 0) return;
        SCur c = s_at(b, u0);
        int i = 0;
        for (int u = u0; u < u1; ++u, ++i) {
            const int s = i % SX;
            if (i >= SX && (!mbar_wait(&bar.empty_x[s], uint32_t(i / SX - 1) & 1u, ctl, b.err) || aborted(ctl))) break;
            const CUtensorMap *map = &b.g[c.gi].tx;
            mbar_expect_tx(&bar.full_x[s], C::kX);
            tma_2d_keep(xbase + uint32_t(s * C::kX), map, 128 * c.kg, 0, &bar.full_x[s]);
            tma_2d_keep(xbase + uint32_t(s * C::kX + MP * 128), map, 128 * c.kg + 64, 0, &bar.full_x[s]);
            s_next(b, c);
        }
        if (aborted(ctl))
            for (int k = i > SX ? i - SX : 0; k < i; ++k) mbar_drain(&bar.full_x[k % SX], uint32_t(k / SX) & 1u, ctl->limit_ns);
        return;
    }

    if (warp >= kIssueWarp) {
        // ------------------------------------------------------------- issuers
        const int t = warp - kIssueWarp;
        if (lane == 0) {
            const uint32_t idesc = umma_idesc(false, MP, false);
            const uint32_t sum = tmem + uint32_t(t * MP);
            SCur c = s_at(b, u0);
            int i = 0;
            for (int u = u0, part = 0; u < u1; ++part) {
                const Fp4One &g = b.g[c.gi];
                const int end = min(u1, g.ubase + (c.nb + 1) * g.KG), ub = min(end, u + kSpan);
                // the sums of the part before have been read
                if (part > 0) mbar_wait(&bar.sum_empty[t], uint32_t(part - 1) & 1u, ctl, b.err);
                tmem_fence_after();
                for (bool fresh = true; u < ub; ++u, ++i) {
                    const int s = i % SX, a = i & 1;
                    mbar_wait(&bar.full_x[s], uint32_t(i / SX) & 1u, ctl, b.err);
                    mbar_wait(&bar.a_full[t][a], uint32_t(i >> 1) & 1u, ctl, b.err);
                    tmem_fence_after();
                    const uint64_t x0 = umma_desc_k(xbase + uint32_t(s * C::kX));
                    const uint32_t ta = tmem + C::kA + uint32_t(2 * t + a) * 64u;
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        // box ks / 4 (half of the k), 16 k = 32 bytes a step inside the swizzle atom
                        umma_tmem_a(sum, ta + 8u * uint32_t(ks), x0 + uint64_t(((ks >> 2) * MP * 128 + 32 * (ks & 3)) >> 4), idesc,
                                    fresh && ks == 0 ? 0u : 1u);
                    }
                    fresh = false;
                    umma_arrive(&bar.a_empty[t][a]);
                    umma_arrive(&bar.empty_x[s]);
                }
                umma_arrive(&bar.sum_full[t]);
                if (u == end) s_next_tile(b, c);
            }
            // every UMMA has completed, and the other warps are done with the memory, before it is
            // freed (also after a timeout, when they run on without waiting)
            umma_arrive(&bar.fin[t]);
            mbar_drain(&bar.fin[t], 0u, ctl->limit_ns);
            mbar_drain(&bar.out, 0u, ctl->limit_ns);
        }
        __syncwarp();
        // both issuers are done
        asm volatile("bar.sync 2, 64;" ::: "memory");
        if (warp == kIssueWarp) {
            tmem_fence_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
        }
        return;
    }

    // ------------------------------------------------------------------ expansion
    const int grp = warp >> 3, h = (warp >> 2) & 1;
    const int t = grp;                                        // the tile whose sums the warp reads
    const int r = 32 * (warp & 3) + lane, col = 128 * t + r;  // row of a tile = lane of the tensor memory
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    // of tile 0 (tile 1: 128 columns on, the same chunk order)
    const uint32_t p0 = uint32_t(r * 64 + 16 * fp4_chunk_at(r, 2 * h)), p1 = uint32_t(r * 64 + 16 * fp4_chunk_at(r, 2 * h + 1));
    const uint32_t ps = uint32_t(kFp4Scales + 8 * r + 4 * h);  // (chunks 2 h and 2 h + 1: k 16 j .. and 64 + 16 j ..)
    const int M = b.M;
    SCur c = s_at(b, u0);
    const int m0 = h * (MP / 2), left = min(M - m0, MP / 2);  // the tokens whose sums the warp reads
    int i = 0, part = 0;
    for (int u = u0; u < u1;) {
        const Fp4One &g = b.g[c.gi];
        const int nb = c.nb, first = g.ubase + nb * g.KG;
        const int ua = u, ub = min(u1, first + g.KG), iend = i + ub - ua;
        // the piece's place for the fix-up; until its end, the sums of its parts so far
        float *place = b.partial + (size_t(blockIdx.x) * 2 + (ua == u0 ? 0 : 1)) * size_t(M) * kFp4Tile + m0 * kFp4Tile + col;
        bool fresh = true;
        int iu = i + ((i & 1) != grp);  // this group's units
#pragma unroll 1
        for (int next = min(i + kSpan, iend);; next = min(next + kSpan, iend), fresh = false, ++part) {
            for (; iu < next; iu += 2) {
                const int s = iu % SW;
                mbar_wait(&bar.full_w[s], uint32_t(iu / SW) & 1u, ctl, b.err);
                const uint32_t st = wbase + uint32_t(s) * kFp4Unit;
#pragma unroll
                for (int tile = 0; tile < 2; ++tile) {
                    const uint4 c0 = lds128(st + p0 + uint32_t(tile * 128 * 64)), c1 = lds128(st + p1 + uint32_t(tile * 128 * 64));
                    const uint32_t f = lds32(st + ps + uint32_t(tile * 128 * 8));
                    if (tile == 1) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.empty_w[s]);
                    }
                    uint32_t v[32];
                    const uint32_t f0 = fp4_scale2(prmt2(f, 0u, 0x4040u)), f1 = fp4_scale2(prmt2(f, 0u, 0x4141u));
                    const uint32_t f2 = fp4_scale2(prmt2(f, 0u, 0x4242u)), f3 = fp4_scale2(prmt2(f, 0u, 0x4343u));
                    const auto expand = [&](uint32_t w, uint32_t scale, int at) {
                        uint32_t(&to)[4] = *reinterpret_cast<uint32_t(*)[4]>(&v[at]);
                        fp4_expand(w, scale, to);
                    };
                    // columns 16 h ..: k 32 h .. + 31; columns 32 + 16 h ..: k 64 + 32 h ..
                    expand(c0.x, f0, 0), expand(c0.y, f0, 4), expand(c1.x, f2, 8), expand(c1.y, f2, 12);
                    expand(c0.z, f1, 16), expand(c0.w, f1, 20), expand(c1.z, f3, 24), expand(c1.w, f3, 28);
                    if (iu >= 2) mbar_wait(&bar.a_empty[tile][grp], uint32_t((iu >> 1) - 1) & 1u, ctl, b.err);
                    tmem_fence_after();
                    const uint32_t ta = tmem + lanes + C::kA + uint32_t(2 * tile + grp) * 64u + 16u * uint32_t(h);
                    tmem_store16(ta, v);
                    tmem_store16(ta + 32u, v + 16);
                    tmem_wait_st();
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.a_full[tile][grp]);
                }
            }
            if (next == iend) break;
            // ---- a part's sums, out of the way of the next one
            mbar_wait(&bar.sum_full[t], uint32_t(part) & 1u, ctl, b.err);
            tmem_fence_after();
            float *to = place;
#pragma unroll 1
            for (int q = 0; q < left; q += 16, to += 16 * kFp4Tile) {
                uint32_t z[16];
                tmem_load16(tmem + lanes + uint32_t(t * MP + m0 + q), z);
                tmem_wait_ld();
                tmem_landed16(z);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (q + e < left) {
                        if (fresh)
                            __stcg(to + e * kFp4Tile, __uint_as_float(z[e]));
                        else
                            add_to(to + e * kFp4Tile, __uint_as_float(z[e]));
                    }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.sum_empty[t]);
        }
        u = ub, i = iend;
        // ---- the piece's sums: row r, tokens h MP / 2 .. + MP / 2
        mbar_wait(&bar.sum_full[t], uint32_t(part) & 1u, ctl, b.err);
        tmem_fence_after();
        const bool whole = ua == first && ub == first + g.KG;
        const int n = nb * kFp4Tile + col;
        // (rolled: a piece of code that runs once costs an SM 250 cycles per 128 bytes of it)
        const float back = kFp4Back * g.scale;
        const size_t at = size_t(m0) * g.N + n;
        float *yf = static_cast<float *>(g.y) + at;
        __nv_bfloat16 *yb = static_cast<__nv_bfloat16 *>(g.y) + at;
#pragma unroll 1
        for (int q = 0; q < left; q += 16, place += 16 * kFp4Tile) {
            uint32_t z[16];
            tmem_load16(tmem + lanes + uint32_t(t * MP + m0 + q), z);
            tmem_wait_ld();
            tmem_landed16(z);
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(z[e]);
            if (!fresh)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (q + e < left) v[e] += load_back(place + e * kFp4Tile);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] *= back;
            if (g.x_scale)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (q + e < left) v[e] *= g.x_scale[m0 + q + e];
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (q + e < left) place[e * kFp4Tile] = v[e];
            } else if (n < g.N) {
                if (b.y_dtype == W12_F32) {
#pragma unroll
                    for (int e = 0; e < 16; ++e, yf += g.N)
                        if (q + e < left) *yf = v[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e, yb += g.N)
                        if (q + e < left) *yb = __float2bfloat16_rn(v[e]);
                }
            }
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bar.sum_empty[t]);
            if (u >= u1) mbar_arrive(&bar.out);
        }
        if (!whole)
            fp4_fixup(b, g, first, nb, ub - ua, &bar.last, threadIdx.x, kDT);
        ++part;
        s_next_tile(b, c);
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                   const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// x [M][K] bf16 in boxes of 64 k x MP tokens, 128-byte swizzle, tokens past M zeros.
int make_map(CUtensorMap *m, const void *x, int64_t K, int M, int MP) {
    const cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(M)};
    const cuuint64_t strides[1] = {cuuint64_t(K * 2)};
    const cuuint32_t box[2] = {64, cuuint32_t(MP)};
    const cuuint32_t es[2] = {1, 1};
    return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(x), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? W12_OK
               : W12_ERR_CUDA;
}

template <int MP>
int occ_t(int *blocks) {
    if (cudaFuncSetAttribute(fp4_tc_kernel<MP>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(TCfg<MP>::kSmem)) != cudaSuccess)
        return W12_ERR_CUDA;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, fp4_tc_kernel<MP>, kThreads, TCfg<MP>::kSmem) == cudaSuccess
               ? W12_OK
               : W12_ERR_CUDA;
}

}  // namespace

int fp4_tc_occupancy(int variant, int *blocks) {
    switch (variant) {
        case kFp4TcVariant: return occ_t<32>(blocks);
        case kFp4TcVariant + 1: return occ_t<64>(blocks);
        case kFp4TcVariant + 2: return occ_t<128>(blocks);
    }
    return W12_ERR_ARG;
}

int launch_fp4_tc(Fp4Batch &b, int grid, void *stream) {
    if (!encoder()) return W12_ERR_CUDA;
    const int v = fp4_variant(b.M), MP = 32 << (v - kFp4TcVariant);
    for (int i = 0; i < b.count; ++i)
        if (make_map(&b.g[i].tx, b.g[i].x, b.g[i].K, b.M, MP) != W12_OK) return W12_ERR_CUDA;
    switch (v) {
        case kFp4TcVariant: return launch_step(fp4_tc_kernel<32>, grid, kThreads, TCfg<32>::kSmem, 1, stream, b);
        case kFp4TcVariant + 1: return launch_step(fp4_tc_kernel<64>, grid, kThreads, TCfg<64>::kSmem, 1, stream, b);
    }
    return launch_step(fp4_tc_kernel<128>, grid, kThreads, TCfg<128>::kSmem, 1, stream, b);
}

}  // namespace w12
