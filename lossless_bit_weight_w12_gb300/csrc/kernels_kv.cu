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
__device__ __forceinline__ void load4(const void *p, int64_t i, float (&x)[4]) {
    if (DT == W12_F32) {
        const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
        x[0] = bf16_bits_to_float(v.x & 0xFFFFu), x[1] = bf16_bits_to_float(v.x >> 16);
        x[2] = bf16_bits_to_float(v.y & 0xFFFFu), x[3] = bf16_bits_to_float(v.y >> 16);
    }
}

__device__ __forceinline__ uint2 pack4_bf16(const float (&x)[4]) {
    return make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

// One row (a head of a token) per group of DIM / 4 lanes, U rows per group
// in flight.  Rows are ordered by token, then query heads, key heads, value
// heads: consecutive lanes read consecutive memory.
template <int DIM, int XT, int KV, int U>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int GL = DIM / 4;            // lanes per row
    constexpr int RPB = kThreads / GL;     // rows per block and step
    const int gl = threadIdx.x % GL, e = 4 * gl;
    const int nh = a.q_heads + 2 * a.heads;
    const int64_t rows = a.tokens * nh;
    const int h2 = a.rot / 2;
    pdl_launch_dependents();
    pdl_wait_previous();
    for (int64_t base = int64_t(blockIdx.x) * (RPB * U); base < rows; base += int64_t(gridDim.x) * (RPB * U)) {
        float x[U][4];
        int64_t tok[U];
        int32_t hd[U], pos[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = base + u * RPB + threadIdx.x / GL;
            tok[u] = i < rows ? i / nh : -1;
            pos[u] = -1;
            if (tok[u] < 0) continue;
            const int hh = int(i - tok[u] * nh);
            hd[u] = hh;
            const int64_t r = tok[u] / a.T;
            pos[u] = a.kv_len[r] - a.T + int(tok[u] - r * a.T);
            if (hh < a.q_heads)
                load4<XT>(a.q, tok[u] * a.q_stride + int64_t(hh) * DIM + e, x[u]);
            else if (hh < a.q_heads + a.heads)
                load4<XT>(a.k, tok[u] * a.k_stride + int64_t(hh - a.q_heads) * DIM + e, x[u]);
            else
                load4<XT>(a.v, tok[u] * a.v_stride + int64_t(hh - a.q_heads - a.heads) * DIM + e, x[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // a whole group of lanes takes the same branches here
            const int hh = tok[u] < 0 ? 0 : hd[u];
            const bool is_q = hh < a.q_heads, is_v = hh >= a.q_heads + a.heads;
            bool live = tok[u] >= 0 && pos[u] >= 0;
            int64_t slot = 0;
            if (live) {
                const int64_t col = int64_t(pos[u]) >> a.page_log2;
                bool ok = a.rot == 0 || int64_t(pos[u]) < a.rope_positions;
                int32_t pg = 0;
                if (col < a.table_cols) {
                    pg = a.table[(tok[u] / a.T) * a.table_cols + col];
                    ok = ok && pg >= 0 && pg < a.n_pages;
                } else {
                    ok = false;
                }
                if (!ok) {  // reported once per row; nothing of the token is written
                    if (gl == 0) record_error(a.err, W12_ERR_DEVICE);
                    live = false;
                }
                slot = ((int64_t(pg) * a.heads + (is_v ? hh - a.q_heads - a.heads : hh - a.q_heads)) << a.page_log2) +
                       (pos[u] & (a.page - 1));
            }
            float y[4] = {x[u][0], x[u][1], x[u][2], x[u][3]};
            if (a.rot && a.interleaved) {
                if (live && !is_v && e < a.rot) {
                    const float *t = a.rope + int64_t(pos[u]) * a.rot + e / 2;
                    const float2 c = *reinterpret_cast<const float2 *>(t), s = *reinterpret_cast<const float2 *>(t + h2);
                    y[0] = turn_a(x[u][0], x[u][1], c.x, s.x), y[1] = turn_b(x[u][0], x[u][1], c.x, s.x);
                    y[2] = turn_a(x[u][2], x[u][3], c.y, s.y), y[3] = turn_b(x[u][2], x[u][3], c.y, s.y);
                }
            } else if (a.rot) {
                // the partner channels e +- rot/2 sit h2/4 lanes away (rot % 8 == 0)
                const bool low = e < h2;
                const int lane = threadIdx.x & 31;
                const int src = (lane & ~(GL - 1)) + ((low ? gl + h2 / 4 : gl - h2 / 4) & (GL - 1));
                float o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = __shfl_sync(0xFFFFFFFFu, x[u][j], src);
                if (live && !is_v && e < a.rot) {
                    const float *t = a.rope + int64_t(pos[u]) * a.rot + (low ? e : e - h2);
                    const float4 c = *reinterpret_cast<const float4 *>(t), s = *reinterpret_cast<const float4 *>(t + h2);
                    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        y[j] = low ? turn_a(x[u][j], o[j], cc[j], ss[j]) : turn_b(o[j], x[u][j], cc[j], ss[j]);
                }
            }
            if (KV == W12_KV_E4M3) {
                float amax = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
                // fmaxf drops a NaN: a non-finite channel is looked for by itself
                bool bad = !(fabsf(y[0]) <= 3.0e38f && fabsf(y[1]) <= 3.0e38f && fabsf(y[2]) <= 3.0e38f &&
                             fabsf(y[3]) <= 3.0e38f);
#pragma unroll
                for (int off = GL / 2; off >= 1; off >>= 1) {
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
                    bad = __shfl_xor_sync(0xFFFFFFFFu, int(bad), off) || bad;
                }
                if (live && !is_q) {
                    const bool some = amax > kTinyRow && !bad;
                    const float inv = some ? __fdiv_rn(kE4m3Max, amax) : 0.0f;
                    float z[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[j] = some ? __fmul_rn(y[j], inv) : 0.0f;
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(z[0], z[1]), __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(z[2], z[3]), __NV_SATFINITE, __NV_E4M3);
                    uint8_t *cache = static_cast<uint8_t *>(is_v ? a.vc : a.kc);
                    *reinterpret_cast<uint32_t *>(cache + slot * DIM + e) = lo | (hi << 16);
                    if (gl == 0)
                        (is_v ? a.vs : a.ks)[slot] =
                            bad ? __int_as_float(0x7FC00000) : some ? __fdiv_rn(amax, kE4m3Max) : 0.0f;
                }
            } else if (live && !is_q) {
                uint16_t *cache = static_cast<uint16_t *>(is_v ? a.vc : a.kc);
                *reinterpret_cast<uint2 *>(cache + slot * DIM + e) = pack4_bf16(y);
            }
            if (live && is_q)
                *reinterpret_cast<uint2 *>(a.q_out + tok[u] * a.out_stride + int64_t(hh) * DIM + e) = pack4_bf16(y);
        }
    }
}

template <int DIM, int XT, int KV>
int append_t(const AppendArgs &a, int sms, void *stream) {
    constexpr int RPB = kThreads / (DIM / 4);
    const int64_t rows = a.tokens * (a.q_heads + 2 * a.heads);
    // One row per group of lanes while that leaves the GPU room for every
    // block at once (8 blocks of 256 threads per SM), four in flight above.
    if (rows <= int64_t(sms) * 8 * RPB)
        return launch_step(append_kernel<DIM, XT, KV, 1>, int((rows + RPB - 1) / RPB), kThreads, 0, 1, stream, a);
    const int64_t blocks = (rows + 4 * RPB - 1) / (4 * RPB);
    const int64_t cap = int64_t(1) << 30;
    return launch_step(append_kernel<DIM, XT, KV, 4>, int(blocks < cap ? blocks : cap), kThreads, 0, 1, stream, a);
}

// kTok tokens per block: the first kTok threads find their token's request
// (binary search in cu_len) and cache slot, then all threads copy the
// tokens' rows in 16-byte pieces, head-major within a token, so that the
// packed output is written in order.
constexpr int kTok = 16;

template <int DIM, int KV>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a) {
    constexpr int EB = KV == W12_KV_E4M3 ? 16 : 8;  // channels per 16-byte piece of the cache
    constexpr int PPR = DIM / EB;                   // pieces per row
    __shared__ int64_t s_at[kTok];                  // first row of (page, head 0) + row in page; -1: none
    pdl_launch_dependents();
    pdl_wait_previous();
    const int64_t t0 = int64_t(blockIdx.x) * kTok;
    if (threadIdx.x < kTok) {
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
    const int n = int(a.tokens - t0 < kTok ? a.tokens - t0 : kTok) * per * 2;
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

int launch_read(const ReadArgs &a, int dim, int kv, void *stream) {
    const int grid = int((a.tokens + kTok - 1) / kTok);
    const bool q8 = kv == W12_KV_E4M3;
    if (dim == 128)
        return q8 ? launch_step(read_kernel<128, W12_KV_E4M3>, grid, kThreads, 0, 1, stream, a)
                  : launch_step(read_kernel<128, W12_KV_BF16>, grid, kThreads, 0, 1, stream, a);
    return q8 ? launch_step(read_kernel<64, W12_KV_E4M3>, grid, kThreads, 0, 1, stream, a)
              : launch_step(read_kernel<64, W12_KV_BF16>, grid, kThreads, 0, 1, stream, a);
}

}  // namespace w12
