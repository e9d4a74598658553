// fp4_device.cuh -- the 4-bit weight format in registers (include/w12.h).
//
// A word holds the codes of 8 consecutive k of a column, the even k in its low
// half, the odd ones in its high half.  Of a half's four codes (pairs p = 0..3)
// the magnitudes lie at bits 8-6, 5-3, 2-0 and 11-9 and the signs at 15, 12, 14
// and 13, so that a pair comes out as two bf16 numbers with at most two shifts
// and two three-input operations: sign at 15, the two exponent bits and the
// mantissa bit at 8-6.  Read as bf16 that is the code's value times 2^-126 (0.5
// is a subnormal number there, as it is in the code), and one bf16x2 product
// with the scale times 2^116 gives the weight times 2^-10 -- exactly: a code has
// 2 significant bits, a scale 4, and bf16 holds 8.
//
// A scale (e4m3 without its sign, which the codes take over) is stored with 5
// exponent bits, bias 9, and 3 mantissa bits: e4m3's subnormals are normal
// numbers there, so its bf16 form is one shift and one addition.  A zero scale
// is a group of zero codes; 0xAF is NaN.
#pragma once

#include <cstdint>

#include "device_common.cuh"
#include "draft_internal.h"
#include "stream_device.cuh"

namespace w12 {

constexpr float kFp4Back = 1024.0f;  // 2^10, what the weights in registers lack

// The k of code 0 of word q of 16-byte chunk j of a column's 64 bytes.
__host__ __device__ constexpr int fp4_k(int j, int q) { return 64 * (q >> 1) + 16 * j + 8 * (q & 1); }
// The place of the scale of k / 16 = g among a column's 8.
__host__ __device__ constexpr int fp4_scale_at(int g) { return 2 * (g & 3) + (g >> 2); }
// The place of chunk j among a column's four.
__host__ __device__ constexpr int fp4_chunk_at(int col, int j) { return j ^ ((col >> 1) & 3); }

// bf16x2 of a scale byte (both halves), times 2^116.
__device__ __forceinline__ uint32_t fp4_scale2(uint32_t byte2) {  // the byte in both halves
    return byte2 * 16u + (((127u - 9u + 116u) << 7) * 0x10001u);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The 8 weights of a word, times 2^-10, as bf16 pairs (k0, k0 + 1), ...
__device__ __forceinline__ void fp4_expand(uint32_t w, uint32_t scale2, uint32_t (&out)[4]) {
    constexpr uint32_t kMag = 0x01C001C0u, kSign = 0x80008000u;
    out[0] = w & (kMag | kSign);
    out[1] = (w << 3) & (kMag | kSign);
    out[2] = ((w << 6) & kMag) | ((w << 1) & kSign);
    out[3] = ((w >> 3) & kMag) | ((w << 2) & kSign);
#pragma unroll
    for (int p = 0; p < 4; ++p) out[p] = mul_bf16x2(out[p], scale2);
}

// 8 codes (nibble i: code of k0 + i, bit 3 its sign) as a word of the format.
__device__ __forceinline__ uint32_t fp4_word(uint32_t nibbles) {
    constexpr int mag[4] = {6, 3, 0, 9}, sign[4] = {15, 12, 14, 13};
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t v = nibbles >> (4 * i);
        w |= ((v & 7u) << mag[i >> 1] | ((v >> 3) & 1u) << sign[i >> 1]) << (16 * (i & 1));
    }
    return w;
}

// The units of this CTA.
__device__ __forceinline__ void fp4_units(const Fp4Batch &b, int &u0, int &u1) {
    const int n = b.U / b.grain, G = int(gridDim.x), c = int(blockIdx.x), per = n / G, rem = n % G;
    u0 = sk_unit_begin(c, per, rem) * b.grain;
    u1 = u0 + (per + (c < rem ? 1 : 0)) * b.grain;
}

// Stream-K fix-up, as stream_fixup (stream_device.cuh), for tiles of 256 columns: up
// to 8 pieces' parts are on their way at a time (16 pieces one after the other: 9 us).
template <int O, int P>
__device__ __forceinline__ void fp4_add_pieces(const Fp4Batch &b, const Fp4One &g, int first, int nb, int c0, int c1, int tid,
                                               int nthreads) {
    const int G = int(gridDim.x), per = b.U / G, rem = b.U % G, total = b.M * (kFp4Tile / 4);
    const size_t slot = size_t(b.M) * kFp4Tile;
#pragma unroll 1
    for (int o0 = tid; o0 < total; o0 += O * nthreads) {
        float4 sum[O];
#pragma unroll
        for (int k = 0; k < O; ++k) sum[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int c = c0; c <= c1; c += P) {
            float4 v[P][O];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int from = min(c + p, c1);
                const float4 *part = reinterpret_cast<const float4 *>(
                    b.partial + (size_t(from) * 2 + (sk_unit_begin(from, per, rem) >= first ? 0 : 1)) * slot);
#pragma unroll
                for (int k = 0; k < O; ++k) v[p][k] = __ldcg(part + min(o0 + k * nthreads, total - 1));
            }
#pragma unroll
            for (int p = 0; p < P; ++p)
                if (c + p <= c1)
#pragma unroll
                    for (int k = 0; k < O; ++k)
                        sum[k].x += v[p][k].x, sum[k].y += v[p][k].y, sum[k].z += v[p][k].z, sum[k].w += v[p][k].w;
        }
#pragma unroll
        for (int k = 0; k < O; ++k) {
            const int o = o0 + k * nthreads, m = o / (kFp4Tile / 4), n = nb * kFp4Tile + 4 * (o % (kFp4Tile / 4));
            if (o >= total) break;
            const float r[4] = {sum[k].x, sum[k].y, sum[k].z, sum[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < g.N) store_out(g.y, b.y_dtype, g.N, m, n + e, r[e]);
        }
    }
}

__device__ __forceinline__ void fp4_fixup(const Fp4Batch &b, const Fp4One &g, int first, int nb, int count, int *s_last, int tid,
                                          int nthreads) {
    const int G = int(gridDim.x), per = b.U / G, rem = b.U % G;
    const int c0 = sk_cta_of(first, per, rem), c1 = sk_cta_of(first + g.KG - 1, per, rem);
    __threadfence();
    named_sync(nthreads);
    if (tid == 0) {
        // a split tile starts in one CTA, as its last: that CTA's number names the
        // counter, as many for any matrix, and one workspace serves them all
        uint32_t *arrived = &b.counters[c0];
        const uint32_t old = atomicAdd(arrived, uint32_t(count));
        *s_last = int(old) + count == g.KG;
        if (*s_last) *arrived = 0u;
    }
    named_sync(nthreads);
    if (*s_last) {
        __threadfence();
        if (c1 - c0 < 2)
            fp4_add_pieces<4, 2>(b, g, first, nb, c0, c1, tid, nthreads);
        else
            fp4_add_pieces<1, 8>(b, g, first, nb, c0, c1, tid, nthreads);
    }
    named_sync(nthreads);  // s_last is reused by the next piece
}

}  // namespace w12
