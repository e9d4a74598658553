// kernels_attend.cu -- attention of draft blocks and single tokens over the
// paged cache, the prefix that all requests share read once.
//
// For a query row at position p: s_j = scale q . k_j over its keys j <= p,
// m = max s_j, out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), lse = m +
// log(sum).  One pass over the keys: with a running maximum m, the sum l and
// the output O are rescaled by 2^(m_old - m_new) whenever m grows (scores
// are kept in units of log2).  m, l and O are fp32; the weights enter the
// second product rounded to bf16 (bf16 cache) or fp16 (e4m3 cache), as
// tensor cores take them; l sums the unrounded ones.
//
// The register kernel, for few query rows per key head (the cache stream
// bounds it) and for every tile that needs a mask: one CTA
// per SM, a producer warp keeps a ring of key/value tiles full with TMA
// boxes (a box per page and tile; 128-byte swizzle, so that the fragment
// loads below have no bank conflicts), 8 consumer warps in two groups take
// alternate tiles, and within a group warp w owns 16 of a tile's 64 keys for
// all query rows: no warp waits for another until a segment ends, when the 8
// (m, l, O) are added up in warp order.  Products are mma.sync m16n8k16 with
// fp32 accumulation.
//
// e4m3 tiles stay 8 bits wide up to the registers: codes are exact in fp16,
// so both products run in fp16; the query row is scaled by a power of two to
// below 2 (its bf16 values then lose nothing that matters: what is 2^-14 of
// the row's largest keeps fewer bits), the key's scale multiplies the score
// and the value's scale the weight.  m only has to keep the exponentials in
// range: with value scales below 2^e it is max - 7 + e, so that weights times
// scales stay below 2^7 and the fp16 they are rounded to is far from both of
// its ends.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "attend_device.cuh"
#include "device_common.cuh"

namespace w12 {

namespace {

constexpr int kCW = 8;                  // consumer warps, two groups of 4
constexpr int kCT = kCW * 32;
constexpr int kAT = kCT + 32;           // + the producer warp
constexpr int kJoinCols = 32;           // channels per step of the CTA's join
constexpr int kJoinPitch = kJoinCols + 4;
constexpr float kNegInf = -INFINITY;

template <int D, bool Q8, int MT>
struct ACfg {
    static constexpr int RT = 16 * MT;
    static constexpr int kTileBytes = AttStage<D, Q8>::kTile;
    static constexpr int kScaleOff = AttStage<D, Q8>::kScale;
    static constexpr int kStage = AttStage<D, Q8>::kBytes;
    static constexpr int kQ = RT * D * 2;
    static constexpr int kJoin = kCW * 16 * kJoinPitch * 4;
    static constexpr int kRowStat = kCW * RT * 8;
    static constexpr int kLens = int(sizeof(AttShared));
    static constexpr int kMisc = 1024;                              // barriers, wait state, scalars
    static constexpr int kFixed = kQ + kJoin + kRowStat + kLens + kMisc;
    static constexpr int kFit = (227 * 1024 - kFixed) / kStage;
    // an even number of stages: a stage is then always the same group's, so
    // one barrier per stage sees its phases one by one
    static constexpr int S = (kFit > 12 ? 12 : kFit) & ~1;
    static constexpr size_t kSmem = size_t(S) * kStage + kFixed;
    static_assert(S >= 2 && kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float2 lds_f2(uint32_t addr) {
    float2 r;
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(r.x), "=f"(r.y) : "r"(addr));
    return r;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr));
    return r;
}

__device__ __forceinline__ void sts_zero16(uint32_t addr) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(addr), "r"(0u) : "memory");
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(addr));
    return r;
}

// Shared-memory address of 16-byte piece c of row `key` of a tile, as the
// TMA boxes lay it: bf16 rows of 128 channels are two 128-byte halves (all
// rows of the first, then of the second); 64-byte rows (e4m3, 64 channels)
// use the 64-byte swizzle.
template <int D, bool Q8>
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int key, int c) {
    if (Q8 && D == 64) return base + uint32_t(key * 64 + ((c ^ ((key >> 1) & 3)) << 4));
    return base + uint32_t((c >> 3) * kAttTile * 128 + key * 128 + (((c & 7) ^ (key & 7)) << 4));
}

// Channel of output register (t, c) of lane quad position q4: the bf16 tiles
// are read with the plain order; an e4m3 lane reads 16 (or 8) neighbouring
// channels of a value row at once, and channel number t of them serves
// product step t.
template <int D, bool Q8>
__device__ __forceinline__ int out_channel(int t, int q4, int c) {
    const int n = 2 * q4 + c;
    if (!Q8) return 8 * t + n;
    if (D == 128) return 16 * n + t;
    return 16 * (n & 3) + 8 * (n >> 2) + t;
}

// Where channel d of a query row goes in the row's shared-memory copy, so
// that the fragment of product step s holds the channels that an e4m3 lane
// has in word s of its key pieces (bf16: as it is).
template <bool Q8>
__device__ __forceinline__ int query_column(int d) {
    if (!Q8) return d;
    const int ch = d >> 4, rem = d & 15, e = rem & 3;
    const int s = 4 * (ch >> 2) + (rem >> 2);
    return 16 * s + 8 * (e >> 1) + 2 * (ch & 3) + (e & 1);
}

template <int D>
__device__ __forceinline__ uint32_t query_at(uint32_t base, int row, int c) {
    return base + uint32_t(row * D * 2 + ((c ^ (row & 7)) << 4));
}

template <int D, bool Q8, int MT>
__global__ void __launch_bounds__(kAT, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
    using C = ACfg<D, Q8, MT>;
    constexpr int S = C::S, RT = C::RT, NT = D / 8, KS = D / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t ring = smem_addr(smem);
    unsigned char *fixed = smem + size_t(S) * C::kStage;
    const uint32_t qs = smem_addr(fixed);
    float *join = reinterpret_cast<float *>(fixed + C::kQ);
    float2 *rowstat = reinterpret_cast<float2 *>(fixed + C::kQ + C::kJoin);
    AttShared &sh = *reinterpret_cast<AttShared *>(fixed + C::kQ + C::kJoin + C::kRowStat);
    unsigned char *misc = fixed + C::kQ + C::kJoin + C::kRowStat + C::kLens;
    misc = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(misc) + 15) & ~uintptr_t(15));
    uint64_t *full = reinterpret_cast<uint64_t *>(misc), *empty = full + S;
    WaitCtl &ctl = *reinterpret_cast<WaitCtl *>(empty + S);
    float *row_m = reinterpret_cast<float *>(misc + 512);  // [RT] the segment's maxima (RT <= 32)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (ring & 1023u) {  // the swizzled boxes need a 1024-byte aligned ring
        if (threadIdx.x == 0) record_error(a.err, W12_ERR_DEVICE);
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kCW / 2);
        }
        ctl.abort = 0;
        ctl.limit_ns = a.wait_ns ? a.wait_ns : kWaitLimitNs;
        mbar_fence_init();
    }
    pdl_launch_dependents();
    pdl_wait_previous();

    const AttPlan plan = att_plan(a, sh, kAT);
    const AttendLine &ln = a.line[a.self];
    const int t0 = plan.t0, t1 = plan.t1;
    if (warp == kCW) {
        att_producer<D, Q8, S>(a, plan, sh, ring, full, empty, &ctl);
        return;
    }

    // ------------------------------------------------------------ consumers
    const int grp = warp >> 2, kw = 16 * (warp & 3);  // this warp's keys of its group's tiles
    const int g8 = lane >> 2, q4 = lane & 3;
    const int r0 = lane & 7, mat = lane >> 3;         // ldmatrix: this lane's row and matrix
    for (int t = t0; t < t1;) {
        const AttSeg seg = att_locate(a, plan, sh, t);
        const int n_tiles = min(seg.left, t1 - t);
        // ---- query rows into shared memory (rows past the unit: zeros)
        named_sync(kCT);  // the previous segment's copy is no longer read
        for (int i = threadIdx.x; i < RT * (D / 8); i += kCT) {
            const int row = i / (D / 8), c = i % (D / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < seg.nrows) {
                const int rho = seg.row0 + row, tok = rho / a.G, hq = seg.head * a.G + rho - tok * a.G;
                v = *reinterpret_cast<const uint4 *>(a.q + tok * a.q_stride + int64_t(hq) * D + 8 * c);
            }
            if (!Q8) {
                const uint32_t at = query_at<D>(qs, row, c);
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                             : "memory");
            } else {
                // the row's largest magnitude (the D / 8 lanes of a row are neighbours)
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
#pragma unroll
                for (int o = 1; o < D / 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                // 2^-e with e the exponent of the largest (kept in [-100, 126])
                int e = int(top >> 7) - 127;
                e = max(-100, min(126, e));
                const float down = __uint_as_float(uint32_t(127 - e) << 23);
                if (c == 0) rowstat[row].x = __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t p = pack_f16(bf16_bits_to_float(w[j] & 0xFFFFu) * down,
                                                bf16_bits_to_float(w[j] >> 16) * down);
                    const int col = query_column<Q8>(8 * c + 2 * j);
                    const uint32_t at = query_at<D>(qs, row, col >> 3) + uint32_t(col & 7) * 2u;
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(p) : "memory");
                }
            }
        }
        named_sync(kCT);
        float up[MT][2];  // per row: scale in log2 units (times the query row's power of two)
        int pos[MT][2];
        int min_pos = 0x7FFFFFFF;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = 16 * m + 8 * h + g8;
                up[m][h] = a.scale_log2 * (Q8 ? rowstat[row].x : 1.0f);
                pos[m][h] = 0x7FFFFFFF;  // rows past the unit: their results are not kept
                if (row < seg.nrows) {
                    const int tok = (seg.row0 + row) / a.G, r = tok / a.T;
                    pos[m][h] = sh.lens[r] - a.T + tok - r * a.T;
                }
                min_pos = min(min_pos, pos[m][h]);
            }
        min_pos = __reduce_min_sync(0xFFFFFFFFu, min_pos);
        if (Q8) named_sync(kCT);  // rowstat is read above and written again at the segment's end

        float o[MT][NT][4];
        float m_run[MT][2], l_run[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            m_run[m][0] = m_run[m][1] = kNegInf;
            l_run[m][0] = l_run[m][1] = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n) o[m][n][0] = o[m][n][1] = o[m][n][2] = o[m][n][3] = 0.0f;
        }

        const int i0 = t - t0;
        for (int k = ((i0 & 1) != grp); k < n_tiles; k += 2) {
            const int i = i0 + k, s = i % S;
            mbar_wait(&full[s], uint32_t(i / S) & 1u, &ctl, a.err);
            const uint32_t kb = ring + uint32_t(s) * uint32_t(C::kStage), vb = kb + uint32_t(C::kTileBytes);
            const int key0 = seg.key(k) + kw;  // this warp's first key
            const bool whole = key0 >= seg.key_begin && key0 + 16 <= seg.key_end && key0 + 15 <= min_pos;

            // ---- scores of 16 keys
            float sc[MT][2][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < 2; ++n) sc[m][n][0] = sc[m][n][1] = sc[m][n][2] = sc[m][n][3] = 0.0f;
            if (Q8) {
                // a lane's pieces of keys g8 and g8 + 8: q4 and, for 128 channels, q4 + 4
                uint4 kx[2][D / 64];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int p = 0; p < D / 64; ++p) kx[n][p] = lds128(tile_at<D, Q8>(kb, kw + 8 * n + g8, q4 + 4 * p));
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t w[2];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const uint4 &x = kx[n][ks >> 2];
                        w[n] = (ks & 3) == 0 ? x.x : (ks & 3) == 1 ? x.y : (ks & 3) == 2 ? x.z : x.w;
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        uint32_t qf[4];
                        ldsm4(qf, query_at<D>(qs, 16 * m + r0 + 8 * (mat & 1), 2 * ks + (mat >> 1)));
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            mma16816<true>(sc[m][n], qf, e4m3x2_lo_to_f16x2(w[n]), e4m3x2_hi_to_f16x2(w[n]));
                    }
                }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t kf[4];
                    ldsm4(kf, tile_at<D, Q8>(kb, kw + 8 * (mat >> 1) + r0, 2 * ks + (mat & 1)));
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        uint32_t qf[4];
                        ldsm4(qf, query_at<D>(qs, 16 * m + r0 + 8 * (mat & 1), 2 * ks + (mat >> 1)));
                        mma16816<false>(sc[m][0], qf, kf[0], kf[1]);
                        mma16816<false>(sc[m][1], qf, kf[2], kf[3]);
                    }
                }
            }
            float2 kscale[2], vscale[2];
            float lift = 0.0f;  // e4m3: e - 7 for value scales below 2^e
            if (Q8) {
                const uint32_t sb = kb + uint32_t(C::kScaleOff) + uint32_t(kw + 2 * q4) * 4u;
                float top = 0.0f;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    kscale[n] = lds_f2(sb + 32u * uint32_t(n));
                    vscale[n] = lds_f2(sb + kAttTile * 4u + 32u * uint32_t(n));
                    // scales of rows that are not the unit's may be anything
                    const int j = key0 + 8 * n + 2 * q4;
                    if (j < seg.key_begin || j >= seg.key_end) kscale[n].x = vscale[n].x = 0.0f;
                    if (j + 1 < seg.key_begin || j + 1 >= seg.key_end) kscale[n].y = vscale[n].y = 0.0f;
                    top = fmaxf(top, fmaxf(vscale[n].x, vscale[n].y));
                }
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                lift = exp_above(top) - 7.0f;
            }
            // ---- mask, running maximum, weights
            uint32_t pf[MT][4];
            float pw[MT][2][4];
            bool moved = false;
            float alpha[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float mx = kNegInf;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float x = sc[m][n][2 * h + c] * up[m][h];
                            if (Q8) x *= c ? kscale[n].y : kscale[n].x;
                            const int j = key0 + 8 * n + 2 * q4 + c;
                            if (!whole && (j < seg.key_begin || j >= seg.key_end || j > pos[m][h])) x = kNegInf;
                            sc[m][n][2 * h + c] = x;
                            mx = fmaxf(mx, x);
                        }
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                    const float mn = fmaxf(m_run[m][h], mx + lift);
                    const float mu = mn == kNegInf ? 0.0f : mn;  // a row without keys so far
                    alpha[m][h] = ex2(m_run[m][h] - mu);
                    moved = moved || m_run[m][h] != mn;
                    m_run[m][h] = mn;
                    float sum = 0.0f;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float p = ex2(sc[m][n][2 * h + c] - mu);
                            sum += p;
                            // a masked weight is zero whatever the key's scale holds
                            pw[m][n][2 * h + c] =
                                !Q8 ? p : p == 0.0f ? 0.0f : p * (c ? vscale[n].y : vscale[n].x);
                        }
                    l_run[m][h] = l_run[m][h] * alpha[m][h] + sum;
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        pf[m][2 * n + h] = Q8 ? pack_f16(pw[m][n][2 * h], pw[m][n][2 * h + 1])
                                              : pack_bf16(pw[m][n][2 * h], pw[m][n][2 * h + 1]);
            }
            if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[m][n][c] *= alpha[m][c >> 1];
            }
            // ---- value rows that some query row must not see
            if (!whole) {
                bool touched = false;
                // rows outside the unit's keys (another request's, or never
                // written) are taken as zeros: 0 * NaN would reach the sum
#pragma unroll 1
                for (int x = lane; x < 16 * (D / (Q8 ? 16 : 8)); x += 32) {
                    const int kr = x / (D / (Q8 ? 16 : 8)), c = x % (D / (Q8 ? 16 : 8)), j = key0 + kr;
                    if (j >= seg.key_end || j < seg.key_begin) {
                        sts_zero16(tile_at<D, Q8>(vb, kw + kr, c));
                        touched = true;
                    }
                }
                // keys that only some rows see: a channel that is not finite
                // is kept out of the matrix product and added to the rows
                // that see it by itself
                uint32_t odd = 0;
#pragma unroll 1
                for (int kr = 0; kr < 16; ++kr) {
                    const int j = key0 + kr;
                    if (j < seg.key_begin || j >= seg.key_end || j <= min_pos) continue;
                    bool bad = false;
                    if (lane < D / (Q8 ? 16 : 8)) {
                        const uint4 x = lds128(tile_at<D, Q8>(vb, kw + kr, lane));
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (Q8)
#pragma unroll
                                for (int b = 0; b < 4; ++b) bad = bad || ((w[e] >> (8 * b)) & 0x7Fu) == 0x7Fu;
                            else
                                bad = bad || (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
                    }
                    if (__any_sync(0xFFFFFFFFu, bad)) odd |= 1u << kr;
                }
                while (odd) {
                    const int kr = __ffs(odd) - 1, j = key0 + kr;
                    odd &= odd - 1u;
                    const int src = (lane & ~3) | ((kr & 7) >> 1);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float w0 = __shfl_sync(0xFFFFFFFFu, kr >= 8 ? pw[m][1][2 * h] : pw[m][0][2 * h], src);
                            const float w1 =
                                __shfl_sync(0xFFFFFFFFu, kr >= 8 ? pw[m][1][2 * h + 1] : pw[m][0][2 * h + 1], src);
                            if (j <= pos[m][h]) {
                                const float p = (kr & 1) ? w1 : w0;
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int c = 0; c < 2; ++c) {
                                        const int d = out_channel<D, Q8>(n, q4, c);
                                        float v;
                                        if (Q8) {
                                            const uint32_t b = lds_u8(tile_at<D, Q8>(vb, kw + kr, d >> 4) + uint32_t(d & 15));
                                            float f[4];
                                            e4m3x4_to_float(b, f);
                                            v = f[0];
                                        } else {
                                            v = bf16_bits_to_float(
                                                lds_u16(tile_at<D, Q8>(vb, kw + kr, d >> 3) + uint32_t(d & 7) * 2u));
                                        }
                                        o[m][n][2 * h + c] += p * v;
                                    }
                            }
                        }
                    __syncwarp();
                    if (lane < D / (Q8 ? 16 : 8)) sts_zero16(tile_at<D, Q8>(vb, kw + kr, lane));
                    touched = true;
                }
                if (touched) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next box lands here
                __syncwarp();
            }
            // ---- weights times values
            if (Q8) {
                const int ka = kw + 2 * q4;
                constexpr int W = D == 128 ? 4 : 2;  // words of a lane's piece of a value row
                uint32_t vx[4][W];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = ka + (j & 1) + 8 * (j >> 1);
                    if (D == 128) {
                        const uint4 x = lds128(tile_at<D, Q8>(vb, key, g8));
                        vx[j][0] = x.x, vx[j][1] = x.y, vx[j][W - 2] = x.z, vx[j][W - 1] = x.w;
                    } else {
                        const uint2 x = lds64(tile_at<D, Q8>(vb, key, g8 & 3) + 8u * uint32_t(g8 >> 2));
                        vx[j][0] = x.x, vx[j][1] = x.y;
                    }
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const uint32_t x0 = prmt2(vx[0][w], vx[1][w], 0x5140u), x1 = prmt2(vx[0][w], vx[1][w], 0x7362u);
                    const uint32_t y0 = prmt2(vx[2][w], vx[3][w], 0x5140u), y1 = prmt2(vx[2][w], vx[3][w], 0x7362u);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t b0 = (e & 1) ? e4m3x2_hi_to_f16x2(e & 2 ? x1 : x0) : e4m3x2_lo_to_f16x2(e & 2 ? x1 : x0);
                        const uint32_t b1 = (e & 1) ? e4m3x2_hi_to_f16x2(e & 2 ? y1 : y0) : e4m3x2_lo_to_f16x2(e & 2 ? y1 : y0);
#pragma unroll
                        for (int m = 0; m < MT; ++m) mma16816<true>(o[m][4 * w + e], pf[m], b0, b1);
                    }
                }
            } else {
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t vf[4];
                    ldsm4t(vf, tile_at<D, Q8>(vb, kw + r0 + 8 * (mat & 1), n + (mat >> 1)));
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma16816<false>(o[m][n], pf[m], vf[0], vf[1]);
                        mma16816<false>(o[m][n + 1], pf[m], vf[2], vf[3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }

        // ---- the segment's end: add up the 8 warps' (m, l, O) in warp order
        const int slot = seg.unit + int(blockIdx.x);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float l = l_run[m][h];
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
                if (q4 == 0) rowstat[warp * RT + 16 * m + 8 * h + g8] = make_float2(m_run[m][h], l);
            }
        named_sync(kCT);
        if (threadIdx.x < RT) {
            const int row = threadIdx.x;
            float m = kNegInf;
#pragma unroll
            for (int w = 0; w < kCW; ++w) m = fmaxf(m, rowstat[w * RT + row].x);
            const float mu = m == kNegInf ? 0.0f : m;
            float l = 0.0f;
#pragma unroll
            for (int w = 0; w < kCW; ++w) l += rowstat[w * RT + row].y * ex2(rowstat[w * RT + row].x - mu);
            row_m[row] = mu;
            if (row < seg.nrows) ln.part_ml[size_t(slot) * RT + row] = make_float2(m, l);
        }
        named_sync(kCT);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                f[h] = ex2(m_run[m][h] - row_m[16 * m + 8 * h + g8]);
#pragma unroll
            for (int c0 = 0; c0 < NT / 4; ++c0) {
                // 32 channels of 16 rows per step: this warp's registers (n, c)
                // of the step, at column 8 (n % 4) + 2 q4 + c
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<float2 *>(&join[(warp * 16 + 8 * h + g8) * kJoinPitch + 8 * n + 2 * q4]) =
                            make_float2(o[m][4 * c0 + n][2 * h] * f[h], o[m][4 * c0 + n][2 * h + 1] * f[h]);
                named_sync(kCT);
                for (int i = threadIdx.x; i < 16 * kJoinCols; i += kCT) {
                    const int row = i / kJoinCols, col = i % kJoinCols;
                    float x = 0.0f;
#pragma unroll
                    for (int w = 0; w < kCW; ++w) x += join[(w * 16 + row) * kJoinPitch + col];
                    const int d = out_channel<D, Q8>(4 * c0 + (col >> 3), (col >> 1) & 3, col & 1);
                    if (16 * m + row < seg.nrows) ln.part_o[(size_t(slot) * RT + 16 * m + row) * D + d] = x;
                }
                named_sync(kCT);
            }
        }
        t += n_tiles;
    }
}

// One warp per output row: the results of its segments in every line, under
// the prefix and of its request, each from the first CTA to the last.
template <int D>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait_previous();
    const int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (i >= int64_t(a.rows) * a.heads) return;
    const int tok = int(i / (a.G * a.heads)), hq = int(i - int64_t(tok) * (a.G * a.heads));
    const int head = hq / a.G, rho = tok * a.G + (hq - head * a.G), r = tok / a.T, in_req = rho - r * a.T * a.G;
    // running maximum of the references, sum and output so far
    float m = kNegInf, l = 0.0f, acc[V] = {};
    const auto add = [&](const AttendLine &ln, int first, int n, int row) {
        // entries (slot, half) first .. : reference and sum of up to 32 at once, a lane each
        for (int k0 = 0; k0 < n * ln.halves; k0 += 32) {
            const int left = min(32, n * ln.halves - k0);
            const size_t e0 = size_t(first) * ln.halves + k0;
            float2 ml = make_float2(kNegInf, 0.0f);
            if (lane < left) ml = ln.part_ml[(e0 + lane) * ln.rt + row];
            float top = ml.x;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const float mn = fmaxf(m, top), mu = mn == kNegInf ? 0.0f : mn;
            const float down = ex2(m - mu);
            l *= down;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] *= down;
            m = mn;
            const float f = ex2(ml.x - mu), lf = ml.y * f;
#pragma unroll 8
            for (int k = 0; k < left; ++k) {
                const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
                const float lk = __shfl_sync(0xFFFFFFFFu, lf, k);
                l += lk;
                // (an entry without keys may hold anything)
                if (fk == 0.0f && lk == 0.0f) continue;
                const float *src = ln.part_o + ((e0 + k) * ln.rt + row) * D + V * lane;
                if (V == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(src);
                    acc[0] += x.x * fk, acc[1] += x.y * fk, acc[V - 2] += x.z * fk, acc[V - 1] += x.w * fk;
                } else {
                    const float2 x = *reinterpret_cast<const float2 *>(src);
                    acc[0] += x.x * fk, acc[1] += x.y * fk;
                }
            }
        }
    };
    for (int q = 0; q < kLines; ++q) {
        const AttendLine &ln = a.line[q];
        if (!ln.grid) continue;
        const int np = ln.plan[0], c_r = ln.plan[1 + r], n_r = ln.plan[2 + r] - c_r;
        const int per_head = ln.pu * np + ln.su * ln.plan[1 + a.R], total = per_head * a.heads;
        const int units = ln.pu + a.R * ln.su;
        if (ln.pu && np) {
            const int p = rho / ln.rt, b = head * per_head + p * np, c = att_owner(total, ln.grid, b);
            add(ln, head * units + p + c, att_owner(total, ln.grid, b + np - 1) - c + 1, rho - p * ln.rt);
        }
        if (ln.su && n_r) {
            const int s = in_req / ln.rt, b = head * per_head + ln.pu * np + ln.su * c_r + s * n_r;
            const int c = att_owner(total, ln.grid, b);
            add(ln, head * units + ln.pu + r * ln.su + s + c, att_owner(total, ln.grid, b + n_r - 1) - c + 1,
                in_req - s * ln.rt);
        }
    }
    const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);  // no key: zeros
    uint16_t *dst = a.out + int64_t(tok) * a.out_stride + int64_t(hq) * D + V * lane;
    if (V == 4)
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[V - 2] * inv, acc[V - 1] * inv));
    else
        *reinterpret_cast<uint32_t *>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
    if (a.lse && lane == 0)
        a.lse[int64_t(tok) * (a.G * a.heads) + hq] =
            l == 0.0f ? kNegInf : ((m == kNegInf ? 0.0f : m) + log2f(l)) * 0.6931471805599453f;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

int cache_map(CUtensorMap *m, void *base, int64_t rows, int dim, bool q8, int box_rows) {
    const int es = q8 ? 1 : 2;
    const cuuint64_t dims[2] = {cuuint64_t(dim), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(dim * es)};
    const cuuint32_t box[2] = {cuuint32_t(q8 ? dim : 64), cuuint32_t(box_rows)};
    const cuuint32_t one[2] = {1, 1};
    return encoder()(m, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, dims, strides,
                     box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     q8 && dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? W12_OK
               : W12_ERR_CUDA;
}

// The dynamic shared-memory limit is raised once per device and variant.
template <int D, bool Q8, int MT>
int run(const AttendArgs &a, void *stream) {
    using C = ACfg<D, Q8, MT>;
    static std::atomic<uint64_t> ready[4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return W12_ERR_CUDA;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(ready[dev >> 6].load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(attend_kernel<D, Q8, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(C::kSmem)) != cudaSuccess)
            return W12_ERR_CUDA;
        ready[dev >> 6].fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_step(attend_kernel<D, Q8, MT>, a.line[a.self].grid, kAT, C::kSmem, 1, stream, a);
}

}  // namespace

int attend_make_maps(AttendArgs &a, const w12_kv *kv) {
    if (!encoder()) return W12_ERR_CUDA;
    const int64_t rows = kv->n_pages * kv->heads * kv->page;
    const int br = kv->page < kAttTile ? kv->page : kAttTile;
    const bool q8 = kv->dtype == W12_KV_E4M3;
    const int st = cache_map(&a.mk, kv->k, rows, kv->head_dim, q8, br);
    return st != W12_OK ? st : cache_map(&a.mv, kv->v, rows, kv->head_dim, q8, br);
}

int launch_attend_rest(const AttendArgs &a, int dim, int kv, void *stream) {
    const bool q8 = kv == W12_KV_E4M3, two = a.line[kLineRest].rt > 16;
    if (dim == 128)
        return q8 ? (two ? run<128, true, 2>(a, stream) : run<128, true, 1>(a, stream))
                  : (two ? run<128, false, 2>(a, stream) : run<128, false, 1>(a, stream));
    return q8 ? (two ? run<64, true, 2>(a, stream) : run<64, true, 1>(a, stream))
              : (two ? run<64, false, 2>(a, stream) : run<64, false, 1>(a, stream));
}

int launch_attend_join(const AttendArgs &a, int dim, void *stream) {
    const int blocks = int((int64_t(a.rows) * a.heads + 7) / 8);
    return dim == 128 ? launch_step(attend_join_kernel<128>, blocks, 256, 0, 1, stream, a)
                      : launch_step(attend_join_kernel<64>, blocks, 256, 0, 1, stream, a);
}

}  // namespace w12
