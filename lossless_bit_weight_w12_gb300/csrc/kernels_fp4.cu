// kernels_fp4.cu -- products with 4-bit weights: y = x W^T, the weights e2m1
// codes with an e4m3 scale for 16 consecutive k and one fp32 number for the
// matrix; their packing into unit blocks, their encoding from bf16.  (More than 16
// tokens: kernels_fp4_tc.cu.)
//
// A step of the product reads every weight once, 0.5625 bytes each, so the
// kernel is a weight stream as the W12 one is: units of 256 columns x 128 k
// (18432 contiguous bytes, one bulk copy), dealt out over the GPU as one line
// (stream-K), a ring of shared-memory stages, split tiles finished by a fix-up
// in CTA order (stream_device.cuh).  The tokens' part of a unit comes through an
// extra warp that reads x some units ahead, turns e4m3 codes into bf16 (exactly)
// and stores it beside the unit's weights.
//
// Eight warps multiply (mma.m16n8k16, weights as operand A): warp w has columns
// 32 w .. 32 w + 31, a lane 32 weights of four of them, expanded in registers
// (fp4_device.cuh).  The tensor core's own sums run over one unit only; they are
// added up in fp32 by the lanes, so their truncation does not pile up.
//
// What bounds it: the instructions of the expansion (some 15 for 8 weights with the
// scale; 67 % of the issue slots) beside the stream, and some 8 us that a call needs whatever
// its size: the first units 1 to 3 us after the start, CTAs that end 3 us apart, the
// fix-up 3.  A layer of 341 M weights (192 MB) at one token 40.5 us, 28.2 for the
// bytes, 33.6 without the expansion, 31.6 without the products besides; 17408 x 5120
// at 8 tokens of e4m3 20.5 us, 7.4 for the bytes.
#include <cuda_runtime.h>

#include "draft_internal.h"
#include "fp4_device.cuh"
#include "step_device.cuh"
#include "stream_device.cuh"

namespace w12 {

namespace {

constexpr int kCW = 8;             // warps that multiply
constexpr int kCT = kCW * 32;
constexpr int kXRow = 256 + 16;    // a token's 128 activations: rows 16 bytes apart in the banks

// NT tiles of 8 tokens.  kAhead: units that the x warp reads ahead of the one it
// stores (a unit's x takes about a microsecond to arrive, the unit's share of the
// weight stream half of one).
template <int NT>
struct FCfg {
    static constexpr int MP = 8 * NT;
    static constexpr int kThreads = (kCW + 2) * 32;
    static constexpr int kPer = 4 * NT;     // 16-byte pieces of bf16 x per lane and unit, at most
    static constexpr int kAhead = NT == 1 ? 3 : 2;
    static constexpr int kStage = kFp4Unit + MP * kXRow;
    static constexpr int kBars = 1024;      // barriers and scalars, after the ring
    static constexpr int S = (227 * 1024 / 2 - 1024 - kBars) / kStage;
    static constexpr size_t kSmem = size_t(S) * kStage + kBars;
    static_assert(S >= 3 && (2 * S) * 8 + 64 <= kBars, "ring");
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void sts128(uint32_t addr, const uint4 &v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(addr));
    return r;
}

// Four e4m3 codes as bf16 pairs.
__device__ __forceinline__ uint2 e4m3x4_to_bf16(uint32_t w) {
    float f[4];
    e4m3x4_to_float(w, f);
    return make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
}

template <int NT, bool E4M3>
__global__ void __launch_bounds__(FCfg<NT>::kThreads, 2) fp4_kernel(const __grid_constant__ Fp4Batch b) {
    using C = FCfg<NT>;
    constexpr int S = C::S;
    extern __shared__ __align__(128) unsigned char smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + size_t(S) * C::kStage);
    uint64_t *empty = full + S;
    WaitCtl &ctl = *reinterpret_cast<WaitCtl *>(empty + S);
    int &s_last = *reinterpret_cast<int *>(empty + S + 2);
    volatile int &s_stored = *(reinterpret_cast<int *>(empty + S + 2) + 1);  // units whose tokens have come, once no more do, + 1
    const uint32_t base = smem_addr(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int M = b.M;
    int u0, u1;
    fp4_units(b, u0, u1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 2);  // the weights' copy (and its bytes), the x warp
            mbar_init(&empty[s], kCW);
        }
        ctl.abort = 0;
        ctl.limit_ns = kWaitLimitNs;
        s_stored = 0;
        mbar_fence_init();
    }
    // the rows past M stay zero
    for (int i = threadIdx.x; i < S * (C::MP - M) * (kXRow / 16); i += C::kThreads) {
        const int s = i / ((C::MP - M) * (kXRow / 16)), at = i % ((C::MP - M) * (kXRow / 16));
        sts128(base + uint32_t(s) * C::kStage + kFp4Unit + uint32_t(M) * kXRow + 16u * uint32_t(at), make_uint4(0, 0, 0, 0));
    }
    __syncthreads();
    if (threadIdx.x == 0) pdl_launch();
    if (u0 >= u1) return;

    if (warp == kCW) {
        // ------------------------------------------------------- weights
        if (lane != 0) return;
        if (!b.early_weights) pdl_wait();
        const uint64_t pol = l2_evict_first_policy();
        SCur c = s_at(b, u0);
        int issued = 0;
        for (int u = u0; u < u1; ++u, ++issued) {
            const int s = issued % S;
            if (issued >= S && (!mbar_wait(&empty[s], uint32_t(issued / S - 1) & 1u, &ctl, b.err) || aborted(&ctl))) break;
            const Fp4One &g = b.g[c.gi];
            mbar_expect_tx(&full[s], kFp4Unit);
            bulk_copy(base + uint32_t(s) * C::kStage, g.units + (size_t(c.nb) * g.KG + c.kg) * kFp4Unit, kFp4Unit, &full[s], pol);
            s_next(b, c);
        }
        // after a timeout: let the copies in flight land, arriving for tokens that will not come
        if (aborted(&ctl)) {
            const uint64_t t0 = global_timer_ns();
            while (!s_stored && global_timer_ns() - t0 < ctl.limit_ns) __nanosleep(1000);
            const int from = issued > S ? issued - S : 0;
            if (s_stored)
                for (int k = max(from, s_stored - 1); k < issued; ++k) mbar_arrive(&full[k % S]);
            for (int k = from; k < issued; ++k) mbar_drain(&full[k % S], uint32_t(k / S) & 1u, ctl.limit_ns);
        }
        return;
    }
    pdl_wait();

    if (warp > kCW) {
        // -------------------------------------------------------- tokens
        constexpr int kPer = E4M3 ? 8 : 16, P = E4M3 ? C::kPer / 2 : C::kPer;  // 16-byte pieces: of a token's part, of a lane's
        uint4 v[C::kAhead][P];
        SCur ahead = s_at(b, u0);
        // unit `ahead`, then the next one (not by the read-only path: the kernel ahead writes x)
        const auto read = [&](uint4(&to)[P]) {
            const Fp4One &g = b.g[ahead.gi];
            const uint8_t *x = static_cast<const uint8_t *>(g.x) + size_t(ahead.kg) * (E4M3 ? 128 : 256);
            const size_t row = size_t(g.K) * (E4M3 ? 1 : 2);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const int p = lane + 32 * q;
                if (p < M * kPer) to[q] = __ldcg(reinterpret_cast<const uint4 *>(x + size_t(p / kPer) * row + 16 * (p % kPer)));
            }
            s_next(b, ahead);
        };
#pragma unroll
        for (int d = 0; d < C::kAhead; ++d)
            if (u0 + d < u1) read(v[d]);
        // (a wait that gave up ends the stores: without waits a second arrival could meet a phase
        // that only waits for its bytes)
        int stored = 0;
        for (int u = u0; u < u1 && stored == u - u0; u += C::kAhead) {
#pragma unroll
            for (int d = 0; d < C::kAhead; ++d) {
                if (u + d >= u1) break;
                const int i = u + d - u0, s = i % S;
                const bool stop = i >= S && (!mbar_wait(&empty[s], uint32_t(i / S - 1) & 1u, &ctl, b.err) || aborted(&ctl));
                if (__any_sync(0xFFFFFFFFu, stop)) break;
                const uint32_t st = base + uint32_t(s) * C::kStage + kFp4Unit;
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    const int p = lane + 32 * q;
                    if (p >= M * kPer) continue;
                    const uint32_t at = st + uint32_t(p / kPer) * kXRow + uint32_t(p % kPer) * (E4M3 ? 32u : 16u);
                    const uint4 &y = v[d][q];
                    if (E4M3) {
                        const uint2 a = e4m3x4_to_bf16(y.x), f = e4m3x4_to_bf16(y.y), e = e4m3x4_to_bf16(y.z), h = e4m3x4_to_bf16(y.w);
                        sts128(at, make_uint4(a.x, a.y, f.x, f.y));
                        sts128(at + 16u, make_uint4(e.x, e.y, h.x, h.y));
                    } else {
                        sts128(at, y);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
                ++stored;
                if (u + d + C::kAhead < u1) read(v[d]);
            }
        }
        if (lane == 0) s_stored = stored + 1;
        return;
    }

    // ------------------------------------------------------------ products
    const int g8 = lane >> 2, t = lane & 3;
    const int ra = 32 * warp + g8;  // tile column of fragment row g8 (and ra + 8, 16, 24: the same chunk order)
    const uint32_t pa = uint32_t(ra * 64 + 16 * fp4_chunk_at(ra, t));
    const uint32_t sa = uint32_t(kFp4Scales + ra * 8 + 2 * t);
    const uint32_t xa = uint32_t(kFp4Unit + g8 * kXRow + 32 * t);  // k 16 t .. of token g8
    SCur c = s_at(b, u0);
    int s = 0;
    uint32_t ph = 0;
    for (int u = u0; u < u1;) {
        const Fp4One &g = b.g[c.gi];
        const int nb = c.nb, first = g.ubase + nb * g.KG;
        const int ua = u, ub = min(u1, first + g.KG);
        float acc[2][NT][4] = {};
        for (; u < ub; ++u) {
            mbar_wait(&full[s], ph, &ctl, b.err);
            const uint32_t st = base + uint32_t(s) * C::kStage;
            uint32_t w[4][4], f[4];  // rows ra + 8 r: codes and scales
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint4 v = lds128(st + pa + uint32_t(r) * 512u);
                w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
                f[r] = lds16(st + sa + uint32_t(r) * 64u);
            }
            float part[2][NT][4] = {};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint4 bx[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) bx[j] = lds128(st + xa + uint32_t(j * 8 * kXRow + 128 * (q >> 1) + 16 * (q & 1)));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // words 0 and 1: the scale of k 16 t .., words 2 and 3: of k 64 + 16 t ..
                    const uint32_t da = fp4_scale2(prmt2(f[2 * h], 0u, q < 2 ? 0x4040u : 0x4141u));
                    const uint32_t db = fp4_scale2(prmt2(f[2 * h + 1], 0u, q < 2 ? 0x4040u : 0x4141u));
                    uint32_t va[4], vb[4];
                    fp4_expand(w[2 * h][q], da, va);
                    fp4_expand(w[2 * h + 1][q], db, vb);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        mma_16816(part[h][j], va[0], vb[0], va[1], vb[1], bx[j].x, bx[j].y);
                        mma_16816(part[h][j], va[2], vb[2], va[3], vb[3], bx[j].z, bx[j].w);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++s == S) s = 0, ph ^= 1u;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[h][j][e] += part[h][j][e];
        }
        // acc[h][j][0..1]: column ra + 16 h, tokens 8 j + 2 t, + 1; [2..3]: column ra + 16 h + 8
        const bool whole = ua == first && ub == first + g.KG;
        float *P = b.partial + (size_t(blockIdx.x) * 2 + (ua == u0 ? 0 : 1)) * size_t(M) * kFp4Tile;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int m = 8 * j + 2 * t + (e & 1), r = ra + 16 * h + (e < 2 ? 0 : 8), n = nb * kFp4Tile + r;
                    if (m >= M) continue;
                    float v = acc[h][j][e] * (kFp4Back * g.scale);
                    if (E4M3) v *= g.x_scale[m];
                    if (!whole)
                        P[m * kFp4Tile + r] = v;
                    else if (n < g.N)
                        store_out(g.y, b.y_dtype, g.N, m, n, v);
                }
        if (!whole)
            fp4_fixup(b, g, first, nb, ub - ua, &s_last, threadIdx.x, kCT);
        s_next_tile(b, c);
    }
}

template <int NT, bool E4M3>
int occ_t(int *blocks) {
    if (cudaFuncSetAttribute(fp4_kernel<NT, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(FCfg<NT>::kSmem)) != cudaSuccess)
        return W12_ERR_CUDA;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, fp4_kernel<NT, E4M3>, FCfg<NT>::kThreads, FCfg<NT>::kSmem) ==
                   cudaSuccess
               ? W12_OK
               : W12_ERR_CUDA;
}

template <int NT>
int launch_t(const Fp4Batch &b, bool e4m3, int grid, void *stream) {
    return launch_step(e4m3 ? fp4_kernel<NT, true> : fp4_kernel<NT, false>, grid, FCfg<NT>::kThreads, FCfg<NT>::kSmem, 1, stream, b);
}

template <int NT>
int occ_nt(int *blocks) {
    int e4m3 = 0;
    if (occ_t<NT, false>(blocks) != W12_OK || occ_t<NT, true>(&e4m3) != W12_OK) return W12_ERR_CUDA;
    if (e4m3 < *blocks) *blocks = e4m3;
    return W12_OK;
}

// ------------------------------------------------------------------ packing

// The unit block place of (column n, 128-k group kg).
__device__ __forceinline__ uint8_t *unit_of(uint8_t *blob, int64_t n, int64_t kg, int64_t KG) {
    return blob + ((n / kFp4Tile) * KG + kg) * kFp4Unit;
}

// Writes column `col` of a unit block: its 16 words of codes (in k order, 8
// codes each) and its 8 scales (e4m3 bytes).
__device__ __forceinline__ void store_column(uint8_t *unit, int col, uint32_t (&words)[16], uint64_t scales) {
    uint64_t kept = 0;
#pragma unroll
    for (int gq = 0; gq < 8; ++gq) {
        const uint32_t s = uint32_t(scales >> (8 * gq)) & 0xFFu, mag = s & 0x7Fu;
        uint32_t byte;
        if (mag == 0x7Fu) {
            byte = 0xAFu;
        } else if (mag >= 8u) {  // exponent e - 7: stored e + 2
            byte = mag + (2u << 3);
        } else if (mag != 0u) {  // mag 2^-9: the leading bit's place above 2^-9
            const int lead = 31 - __clz(mag);
            byte = uint32_t(lead << 3) | ((mag << (3 - lead)) & 7u);
        } else {
            byte = 0u;
            words[2 * gq] = words[2 * gq + 1] = 0u;
        }
        if (s & 0x80u) words[2 * gq] ^= 0x88888888u, words[2 * gq + 1] ^= 0x88888888u;
        kept |= uint64_t(byte) << (8 * fp4_scale_at(gq));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = fp4_word(words[fp4_k(j, q) / 8]);
        *reinterpret_cast<uint4 *>(unit + col * 64 + 16 * fp4_chunk_at(col, j)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint64_t *>(unit + kFp4Scales + 8 * col) = kept;
}

constexpr int kPackThreads = 256;

// A thread per (column, 128-k group); columns past N are zeros.
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const uint8_t *codes, const uint8_t *scales, int64_t KG, int64_t N,
                                                            int64_t NP, uint8_t *blob) {
    const int64_t i = int64_t(blockIdx.x) * kPackThreads + threadIdx.x;
    const int64_t n = i / KG, kg = i % KG;
    if (n >= NP) return;
    uint32_t words[16] = {};
    uint64_t s = 0;
    if (n < N) {
        const uint4 *p = reinterpret_cast<const uint4 *>(codes + (n * KG + kg) * 64);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 v = p[j];
            words[4 * j] = v.x, words[4 * j + 1] = v.y, words[4 * j + 2] = v.z, words[4 * j + 3] = v.w;
        }
        s = *reinterpret_cast<const uint64_t *>(scales + (n * KG + kg) * 8);
    }
    store_column(unit_of(blob, n, kg, KG), int(n % kFp4Tile), words, s);
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    float f[4];
    e4m3x4_to_float(byte, f);
    return f[0];
}

// The nearest e2m1 code of |v| (ties to the even one), 0 .. 7.
__device__ __forceinline__ uint32_t e2m1_code(float a) {
    return (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
}

// The same from bf16 weights [N][K].  A division per group, a product per weight: a
// code's argument is off by three roundings.
__global__ void __launch_bounds__(kPackThreads) encode_kernel(const uint16_t *w, int64_t KG, int64_t N, int64_t NP, float scale,
                                                              uint8_t *blob) {
    const int64_t i = int64_t(blockIdx.x) * kPackThreads + threadIdx.x;
    const int64_t n = i / KG, kg = i % KG;
    if (n >= NP) return;
    uint32_t words[16] = {};
    uint64_t scales = 0;
    if (n < N) {
        const uint4 *p = reinterpret_cast<const uint4 *>(w + (n * KG + kg) * 128);
#pragma unroll
        for (int gq = 0; gq < 8; ++gq) {
            const uint4 a = p[2 * gq], d = p[2 * gq + 1];
            const uint32_t raw[8] = {a.x, a.y, a.z, a.w, d.x, d.y, d.z, d.w};
            float v[16];
            uint32_t top = 0;  // as bits: NaN above infinity
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                v[e] = bf16_bits_to_float((raw[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
                top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
            }
            const float amax = __uint_as_float(top);
            uint32_t s;
            if (amax != amax) {
                s = 0x7Fu;
            } else {
                const float want = __fdiv_rn(amax, 6.0f * scale);
                uint16_t c;
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.0f), "f"(fminf(want, 448.0f)));
                s = c & 0xFFu;
                if (s == 0u && amax > 0.0f) s = 1u;
            }
            const float inv = s == 0u || s == 0x7Fu ? 0.0f : __fdiv_rn(1.0f, e4m3_value(s) * scale);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t c = e2m1_code(fabsf(v[e]) * inv) | (v[e] < 0.0f ? 8u : 0u);
                words[2 * gq + (e >> 3)] |= c << (4 * (e & 7));
            }
            scales |= uint64_t(s) << (8 * gq);
        }
    }
    store_column(unit_of(blob, n, kg, KG), int(n % kFp4Tile), words, scales);
}

// Back to fp32 [N][K]: code times scale (exact) times the matrix's number.
__global__ void __launch_bounds__(kPackThreads) decode_kernel(const uint8_t *blob, int64_t KG, int64_t N, float scale, float *out) {
    const int64_t i = int64_t(blockIdx.x) * kPackThreads + threadIdx.x;
    const int64_t n = i / KG, kg = i % KG;
    if (n >= N) return;
    const uint8_t *unit = unit_of(const_cast<uint8_t *>(blob), n, kg, KG);
    const int col = int(n % kFp4Tile);
    float *o = out + (n * KG + kg) * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 v = *reinterpret_cast<const uint4 *>(unit + col * 64 + 16 * fp4_chunk_at(col, j));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int k = fp4_k(j, q);
            const uint32_t byte = unit[kFp4Scales + 8 * col + fp4_scale_at(k / 16)];
            uint32_t x[4];
            fp4_expand(w[q], fp4_scale2(byte * 0x10001u), x);
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = bf16_bits_to_float((x[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) * kFp4Back * scale;
            *reinterpret_cast<float4 *>(o + k) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4 *>(o + k + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
    }
}

int pack_grid(int64_t columns, int64_t KG, unsigned *grid) {
    const int64_t n = (columns * KG + kPackThreads - 1) / kPackThreads;
    if (n >= (int64_t(1) << 31)) return W12_ERR_SHAPE;
    *grid = unsigned(n);
    return W12_OK;
}

int launched() { return cudaGetLastError() == cudaSuccess ? W12_OK : W12_ERR_CUDA; }

// n16 x 16 codes, 16 a thread.
struct WidenArgs {
    const uint4 *codes;
    uint4 *out;
    int64_t n16;
};
__global__ void __launch_bounds__(256) widen_kernel(const __grid_constant__ WidenArgs a) {
    pdl_launch_dependents();
    pdl_wait_previous();
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= a.n16) return;
    const uint4 y = a.codes[i];
    const uint2 p = e4m3x4_to_bf16(y.x), f = e4m3x4_to_bf16(y.y), e = e4m3x4_to_bf16(y.z), h = e4m3x4_to_bf16(y.w);
    a.out[2 * i] = make_uint4(p.x, p.y, f.x, f.y);
    a.out[2 * i + 1] = make_uint4(e.x, e.y, h.x, h.y);
}

}  // namespace

int launch_fp4_widen(const void *codes, void *out, int64_t n, void *stream) {
    const WidenArgs a{static_cast<const uint4 *>(codes), static_cast<uint4 *>(out), n / 16};
    return launch_step(widen_kernel, int((a.n16 + 255) / 256), 256, 0, 1, stream, a);
}

int launch_fp4_pack(const uint8_t *codes, const uint8_t *scales, int64_t K, int64_t N, void *blob, void *stream) {
    const int64_t NP = (N + kFp4Tile - 1) / kFp4Tile * kFp4Tile, KG = K / kGroup;
    unsigned grid;
    const int st = pack_grid(NP, KG, &grid);
    if (st != W12_OK) return st;
    pack_kernel<<<grid, kPackThreads, 0, static_cast<cudaStream_t>(stream)>>>(codes, scales, KG, N, NP, static_cast<uint8_t *>(blob));
    return launched();
}

int launch_fp4_encode(const uint16_t *w, int64_t K, int64_t N, float scale, void *blob, void *stream) {
    const int64_t NP = (N + kFp4Tile - 1) / kFp4Tile * kFp4Tile, KG = K / kGroup;
    unsigned grid;
    const int st = pack_grid(NP, KG, &grid);
    if (st != W12_OK) return st;
    encode_kernel<<<grid, kPackThreads, 0, static_cast<cudaStream_t>(stream)>>>(w, KG, N, NP, scale, static_cast<uint8_t *>(blob));
    return launched();
}

int launch_fp4_decode(const void *blob, int64_t K, int64_t N, float scale, float *out, void *stream) {
    unsigned grid;
    const int st = pack_grid(N, K / kGroup, &grid);
    if (st != W12_OK) return st;
    decode_kernel<<<grid, kPackThreads, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<const uint8_t *>(blob), K / kGroup, N, scale, out);
    return launched();
}

int fp4_occupancy(int variant, int *blocks) {
    switch (variant) {
        case 0: return occ_nt<1>(blocks);
        case 1: return occ_nt<2>(blocks);
    }
    return fp4_tc_occupancy(variant, blocks);
}

int launch_fp4(const Fp4Batch &b, bool e4m3, int grid, void *stream) {
    return fp4_variant(b.M) == 0 ? launch_t<1>(b, e4m3, grid, stream) : launch_t<2>(b, e4m3, grid, stream);
}

}  // namespace w12
