// kernels_kv.cu -- the paged key/value cache: append with rotary positions
// (and quantisation to e4m3), and read-back.
//
// Rotary positions turn channel pair j of a head at position p by the angle
// a(p, j): (x, y) -> (x cos a - y sin a, y cos a + x sin a).  cos and sin
// come from a table made once in double precision (w12_rope_table), so a
// kernel neither evaluates them nor loses the angle's low bits at long
// positions.  The products and the sum are rounded one by one (no fused
// multiply-add), so that a row's bits do not depend on how a compiler
// contracts the expression; the arithmetic is far from the bound.
//
// Both kernels move bytes: read-back of 128000 e4m3 tokens of 8 heads takes
// 125.6 us for 795 MB (6.3 TB/s), append of 8186 tokens of 48 rows of 64
// channels, bf16 to e4m3, 21.4 us for 94 MB (to bf16 18.7 us for 102 MB); one
// token 1.7 us, the launch.
//
// e4m3 rows carry one fp32 scale per token and head, amax / 448 (448 is
// e4m3's largest value): the row uses the format's whole range, a row's
// error is relative to its own largest value, and nothing is known about
// later tokens when a row is written.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "step_device.cuh"
#include "step_internal.h"

namespace w12 {

namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.0f;
constexpr float kTinyRow = 1e-30f;  // a row of smaller magnitudes is stored as zeros (448 / amax would overflow)

// Four consecutive channels of a row of x as floats.
template <int DT>
__device__ __forceinline__ void load4(const void *p, int64_t i, float *x) {
    if (DT == W12_F32) {
        const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
        x[0] = bf16_bits_to_float(v.x & 0xFFFFu), x[1] = bf16_bits_to_float(v.x >> 16);
        x[2] = bf16_bits_to_float(v.y & 0xFFFFu), x[3] = bf16_bits_to_float(v.y >> 16);
    }
}

// What a lane of the append kernel keeps of its token: 8 channels e .. e + 7,
// two blocks of 4, their rotary cosines and sines (the sign of the turn in
// the sine: y = x cos + partner sin).
struct AppendLane {
    int e, mate[2];  // HALF: where the partners of a block are, relative to it
    bool turned[2];
    float cs[8], sn[8];
    int64_t slot0;   // cache row of head 0
    uint32_t group;  // lanes of the row
};

// Eight channels of a row as they lie in memory.
template <int XT>
struct Raw {
    uint2 v[XT == W12_F32 ? 4 : 2];
};
template <int XT>
__device__ __forceinline__ Raw<XT> load_raw(const unsigned char *p) {
    Raw<XT> r;
    if (XT == W12_F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 x = reinterpret_cast<const uint4 *>(p)[h];
            r.v[2 * h] = make_uint2(x.x, x.y), r.v[2 * h + 1] = make_uint2(x.z, x.w);
        }
    } else {  // (only 8-byte alignment is asked for)
        r.v[0] = reinterpret_cast<const uint2 *>(p)[0], r.v[1] = reinterpret_cast<const uint2 *>(p)[1];
    }
    return r;
}
template <int XT>
__device__ __forceinline__ void unpack(const Raw<XT> &r, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < (XT == W12_F32 ? 4 : 2); ++j) {
        if (XT == W12_F32) {
            x[2 * j] = __uint_as_float(r.v[j].x), x[2 * j + 1] = __uint_as_float(r.v[j].y);
        } else {
            x[4 * j] = bf16_bits_to_float(r.v[j].x & 0xFFFFu), x[4 * j + 1] = bf16_bits_to_float(r.v[j].x >> 16);
            x[4 * j + 2] = bf16_bits_to_float(r.v[j].y & 0xFFFFu), x[4 * j + 3] = bf16_bits_to_float(r.v[j].y >> 16);
        }
    }
}

// One row of head hd (query heads, key heads, value heads in order), src:
// where its channel e is.
template <int DIM, int XT, int KV, bool IL>
__device__ __forceinline__ void append_row(const AppendArgs &a, const AppendLane &ln, const Raw<XT> &raw,
                                           const unsigned char *src, int hd, uint16_t *q_out) {
    constexpr int ES = XT == W12_F32 ? 4 : 2;
    const bool query = hd < a.q_heads, value = hd >= a.q_heads + a.heads;
    float x[8], y[8], o[8];
    unpack<XT>(raw, x);
    if (!IL)
#pragma unroll
        for (int b = 0; b < 2; ++b)
            if (ln.turned[b] && !value) load4<XT>(src + 4 * b * ES, ln.mate[b], o + 4 * b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = x[j];
        if (ln.turned[j / 4] && !value)
            y[j] = __fadd_rn(__fmul_rn(x[j], ln.cs[j]), __fmul_rn(IL ? x[j ^ 1] : o[j], ln.sn[j]));
    }
    const int kh = value ? hd - a.q_heads - a.heads : hd - a.q_heads;
    const int64_t slot = ln.slot0 + (int64_t(kh) << a.page_log2);
    if (KV == W12_KV_BF16 || query) {
        uint16_t *to = query ? q_out + int64_t(hd) * DIM : static_cast<uint16_t *>(value ? a.vc : a.kc) + slot * DIM;
        *reinterpret_cast<uint4 *>(to + ln.e) =
            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        return;
    }
    // the largest magnitude by its bits: an infinity and then a NaN are above
    // every finite one
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(y[j]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(ln.group, top);
    const float amax = __uint_as_float(top);
    const bool bad = top >= 0x7F800000u, some = amax > kTinyRow && !bad;
    const float inv = some ? __fdiv_rn(kE4m3Max, amax) : 0.0f;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(y[2 * j], inv), __fmul_rn(y[2 * j + 1], inv)), __NV_SATFINITE,
                                        __NV_E4M3);
    if (!some) w[0] = w[1] = w[2] = w[3] = 0u;  // (0 times an infinity)
    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(value ? a.vc : a.kc) + slot * DIM + ln.e) =
        make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    if (ln.e == 0)
        (value ? a.vs : a.ks)[slot] = bad ? __int_as_float(0x7FC00000) : some ? __fdiv_rn(amax, kE4m3Max) : 0.0f;
}

// A group of DIM / 8 lanes has one token and every `parts`-th of its rows,
// and reads the token's rotary row and cache slot once -- behind the loads of
// its first rows, which need neither.  rot is a multiple of 8, so a lane's
// block of 4 channels lies in one half of the rotated ones: its pair partners
// are the block rot / 2 further or back (read again, from L1) or, interleaved
// (IL), its own neighbours.
template <int DIM, int XT, int KV, bool IL, int kAhead>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int GL = DIM / 8, ES = XT == W12_F32 ? 4 : 2;
    const uint32_t g = blockIdx.x * uint32_t(kThreads / GL) + threadIdx.x / GL;
    const uint32_t tok = g / uint32_t(a.parts), part = g - tok * uint32_t(a.parts);
    AppendLane ln;
    ln.e = 8 * (threadIdx.x % GL);
    ln.group = ((1u << GL) - 1u) << ((threadIdx.x & 31) / GL * GL);
    pdl_launch_dependents();
    pdl_wait_previous();
    if (tok >= uint32_t(a.tokens)) return;  // (whole groups leave; the reductions are the group's)
    const int rows = a.q_heads + 2 * a.heads;
    const unsigned char *q = static_cast<const unsigned char *>(a.q) + (int64_t(tok) * a.q_stride + ln.e) * ES;
    const unsigned char *k = static_cast<const unsigned char *>(a.k) + (int64_t(tok) * a.k_stride + ln.e) * ES;
    const unsigned char *v = static_cast<const unsigned char *>(a.v) + (int64_t(tok) * a.v_stride + ln.e) * ES;
    const auto source = [&](int hd) {
        const unsigned char *p = hd < a.q_heads ? q : hd < a.q_heads + a.heads ? k : v;
        const int h = hd < a.q_heads ? hd : hd < a.q_heads + a.heads ? hd - a.q_heads : hd - a.q_heads - a.heads;
        return p + int64_t(h) * (DIM * ES);
    };
    Raw<XT> raw[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int hd = int(part) + i * a.parts;
        if (hd < rows) raw[i] = load_raw<XT>(source(hd));
    }
    const uint32_t r = tok / uint32_t(a.T);
    // (a negative length counts as 0: all its tokens are padding)
    const int pos = max(a.kv_len[r], 0) - a.T + int(tok - r * uint32_t(a.T));
    if (pos < 0) return;
    const int64_t col = int64_t(pos) >> a.page_log2;
    const int32_t pg = col < a.table_cols ? a.table[r * a.table_cols + col] : -1;
    if (pg < 0 || pg >= a.n_pages || (a.rot && int64_t(pos) >= a.rope_positions)) {
        if (ln.e == 0) record_error(a.err, W12_ERR_DEVICE);  // nothing of the token is written
        return;
    }
    ln.slot0 = ((int64_t(pg) * a.heads) << a.page_log2) + (pos & (a.page - 1));
    const int h2 = a.rot / 2;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int eb = ln.e + 4 * b;
        const bool low = eb < h2;
        ln.turned[b] = eb < a.rot;
        ln.mate[b] = low ? h2 : -h2;
        if (!ln.turned[b]) continue;
        const float *t = a.rope + int64_t(pos) * a.rot;
        float *c4 = ln.cs + 4 * b, *s4 = ln.sn + 4 * b;
        if (IL) {
            const float2 c = *reinterpret_cast<const float2 *>(t + eb / 2), s = *reinterpret_cast<const float2 *>(t + h2 + eb / 2);
            c4[0] = c4[1] = c.x, c4[2] = c4[3] = c.y;
            s4[0] = -s.x, s4[1] = s.x, s4[2] = -s.y, s4[3] = s.y;
        } else {
            const int j = low ? eb : eb - h2;
            const float4 c = *reinterpret_cast<const float4 *>(t + j), s = *reinterpret_cast<const float4 *>(t + h2 + j);
            c4[0] = c.x, c4[1] = c.y, c4[2] = c.z, c4[3] = c.w;
            s4[0] = low ? -s.x : s.x, s4[1] = low ? -s.y : s.y, s4[2] = low ? -s.z : s.z, s4[3] = low ? -s.w : s.w;
        }
    }
    uint16_t *out = a.q_out + int64_t(tok) * a.out_stride;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int hd = int(part) + i * a.parts;
        if (hd >= rows) return;
        append_row<DIM, XT, KV, IL>(a, ln, raw[i], source(hd), hd, out);
    }
#pragma unroll 1
    for (int hd = int(part) + kAhead * a.parts; hd < rows; hd += a.parts) {
        const unsigned char *src = source(hd);
        append_row<DIM, XT, KV, IL>(a, ln, load_raw<XT>(src), src, hd, out);
    }
}

template <int DIM, int XT, int KV>
int append_t(AppendArgs a, int sms, void *stream) {
    constexpr int64_t GPB = kThreads / (DIM / 8);  // groups per block
    const int64_t nh = a.q_heads + 2 * a.heads;
    // A group per row while all blocks fit the GPU at once (8 blocks of 256
    // threads per SM); else 8 groups a token, which share its rotary row and
    // look-up over nh / 8 rows (8186 tokens of 48 rows of 64: 21.0 us; 4 or 16
    // groups 23.6) and load their first rows ahead of the look-up (without
    // 23.2; with 64 registers, which leaves 4 blocks on an SM).
    a.parts = int32_t(a.tokens * nh <= int64_t(sms) * 8 * GPB ? nh : nh < 8 ? nh : 8);
    if (a.tokens * a.parts >= int64_t(1) << 32) a.parts = 1;
    const int grid = int((a.tokens * a.parts + GPB - 1) / GPB);
    constexpr int kAhead = XT == W12_F32 ? 3 : 6;
    if (a.parts == nh)
        return a.interleaved ? launch_step(append_kernel<DIM, XT, KV, true, 1>, grid, kThreads, 0, 1, stream, a)
                             : launch_step(append_kernel<DIM, XT, KV, false, 1>, grid, kThreads, 0, 1, stream, a);
    return a.interleaved ? launch_step(append_kernel<DIM, XT, KV, true, kAhead>, grid, kThreads, 0, 1, stream, a)
                         : launch_step(append_kernel<DIM, XT, KV, false, kAhead>, grid, kThreads, 0, 1, stream, a);
}

// TOK tokens per block: the first TOK threads find their token's request
// (binary search in cu_len) and cache slot, then all threads copy the
// tokens' rows in 16-byte pieces, head-major within a token, so that the
// packed output is written in order.
template <int DIM, int KV, int TOK>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a) {
    constexpr int EB = KV == W12_KV_E4M3 ? 16 : 8;  // channels per 16-byte piece of the cache
    constexpr int PPR = DIM / EB;                   // pieces per row
    __shared__ int64_t s_at[TOK];                  // first row of (page, head 0) + row in page; -1: none
    pdl_launch_dependents();
    pdl_wait_previous();
    const int64_t t0 = int64_t(blockIdx.x) * TOK;
    if (threadIdx.x < TOK) {
        const int64_t t = t0 + threadIdx.x;
        int64_t at = -1;
        if (t < a.tokens) {
            int64_t lo = 0, hi = a.R;  // the last r with cu_len[r] <= t
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) >> 1;
                if (a.cu_len[mid] <= t) lo = mid; else hi = mid;
            }
            const int64_t p = t - a.cu_len[lo], col = p >> a.page_log2;
            int32_t pg = -1;
            if (p >= 0 && t < a.cu_len[lo + 1] && col < a.table_cols) pg = a.table[lo * a.table_cols + col];
            if (pg >= 0 && pg < a.n_pages)
                at = ((int64_t(pg) * a.heads) << a.page_log2) + (p & (a.page - 1));
            else
                record_error(a.err, W12_ERR_DEVICE);
        }
        s_at[threadIdx.x] = at;
    }
    __syncthreads();
    const int per = a.heads * PPR;  // pieces of k (or v) per token
    const int n = int(a.tokens - t0 < TOK ? a.tokens - t0 : TOK) * per * 2;
    constexpr int U = 4;
    for (int i0 = threadIdx.x; i0 < n; i0 += kThreads * U) {
        uint4 x[U];
        float sc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kThreads;
            x[u] = make_uint4(0, 0, 0, 0);
            sc[u] = 0.0f;
            if (i >= n) continue;
            const int tk = i / (2 * per), w = i - tk * 2 * per, is_v = w >= per, j = is_v ? w - per : w;
            const int64_t at = s_at[tk];
            if (at < 0) continue;
            const int64_t row = at + (int64_t(j / PPR) << a.page_log2);
            x[u] = ldg_stream(static_cast<const uint8_t *>(is_v ? a.vc : a.kc) + (row * PPR + j % PPR) * 16);
            if (KV == W12_KV_E4M3) sc[u] = (is_v ? a.vs : a.ks)[row];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kThreads;
            if (i >= n) continue;
            const int tk = i / (2 * per), w = i - tk * 2 * per, is_v = w >= per, j = is_v ? w - per : w;
            uint16_t *o = (is_v ? a.v_out : a.k_out) + ((t0 + tk) * per + j) * EB;
            if (KV == W12_KV_E4M3) {
                const uint32_t w4[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                uint32_t r[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float f[4];
                    e4m3x4_to_float(w4[q], f);
                    r[2 * q] = pack_bf16(__fmul_rn(f[0], sc[u]), __fmul_rn(f[1], sc[u]));
                    r[2 * q + 1] = pack_bf16(__fmul_rn(f[2], sc[u]), __fmul_rn(f[3], sc[u]));
                }
                reinterpret_cast<uint4 *>(o)[0] = make_uint4(r[0], r[1], r[2], r[3]);
                reinterpret_cast<uint4 *>(o)[1] = make_uint4(r[4], r[5], r[6], r[7]);
            } else {
                *reinterpret_cast<uint4 *>(o) = x[u];
            }
        }
    }
}

template <int DIM, int KV>
int read_t(const ReadArgs &a, int sms, void *stream) {
    // 16 tokens a block; 4 where that leaves SMs idle (850 tokens of 8 heads,
    // bf16: 6.4 us with 16, 4.7 with 4)
    const int tok = a.tokens <= int64_t(sms) * 32 ? 4 : 16;
    const int grid = int((a.tokens + tok - 1) / tok);
    return tok == 4 ? launch_step(read_kernel<DIM, KV, 4>, grid, kThreads, 0, 1, stream, a)
                    : launch_step(read_kernel<DIM, KV, 16>, grid, kThreads, 0, 1, stream, a);
}

}  // namespace

int launch_append(const AppendArgs &a, int xt, int dim, int kv, int sms, void *stream) {
    const bool f32 = xt == W12_F32, q8 = kv == W12_KV_E4M3;
    if (dim == 128)
        return f32 ? (q8 ? append_t<128, W12_F32, W12_KV_E4M3>(a, sms, stream)
                         : append_t<128, W12_F32, W12_KV_BF16>(a, sms, stream))
                   : (q8 ? append_t<128, W12_BF16, W12_KV_E4M3>(a, sms, stream)
                         : append_t<128, W12_BF16, W12_KV_BF16>(a, sms, stream));
    return f32 ? (q8 ? append_t<64, W12_F32, W12_KV_E4M3>(a, sms, stream)
                     : append_t<64, W12_F32, W12_KV_BF16>(a, sms, stream))
               : (q8 ? append_t<64, W12_BF16, W12_KV_E4M3>(a, sms, stream)
                     : append_t<64, W12_BF16, W12_KV_BF16>(a, sms, stream));
}

int launch_read(const ReadArgs &a, int dim, int kv, int sms, void *stream) {
    const bool q8 = kv == W12_KV_E4M3;
    if (dim == 128)
        return q8 ? read_t<128, W12_KV_E4M3>(a, sms, stream) : read_t<128, W12_KV_BF16>(a, sms, stream);
    return q8 ? read_t<64, W12_KV_E4M3>(a, sms, stream) : read_t<64, W12_KV_BF16>(a, sms, stream);
}

}  // namespace w12
