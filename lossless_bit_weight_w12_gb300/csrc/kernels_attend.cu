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
// The register kernel, for requests with few query rows per key head (the cache
// stream bounds it).  One CTA per SM with two
// workers, each four warps with a ring of key/value tiles of its own and its
// own piece of the work: while one finishes a segment the other streams.  A
// warp owns 16 of a tile's 64 keys for all query rows; no warp waits for
// another until a segment ends, when the four (m, l, O) are added up in warp
// order.  Producer warps fill the rings with TMA boxes (a box per page and
// tile; 128-byte swizzle, so that the fragment loads below have no bank
// conflicts).  Products are mma.sync m16n8k16 with fp32 accumulation,
// transposed: S^T = K Q^T has the 16 keys as its rows and the query rows as
// its columns, O^T = V^T P^T the channels as its rows, so that a block of
// query rows is 8 wide and not 16 (48 query heads over 8 key heads make 6
// rows a token); P^T is turned between the two by movmatrix.
//
// What bounds it: the cache stream for long contexts -- one request of 131000
// keys, 8 key heads, e4m3 (277 MB): 55 us, of which 44 stream at 6.3 TB/s --
// and for short ones the fixed parts: plan, first tile, the four warps' sums,
// the add-up of partial results, 2 - 3 us each (4 requests of 300 .. 2500
// keys, bf16: 13.6 us for 23 MB).
//
// e4m3 tiles stay 8 bits wide up to the registers: codes are exact in fp16,
// so both products run in fp16; the query row is scaled by a power of two to
// below 2 (its bf16 values then lose nothing that matters: what is 2^-14 of
// the row's largest keeps fewer bits), the key's scale multiplies the score
// and the value's scale the weight.  m only has to keep the exponentials in
// range: with the value scales that a row sees below 2^e it is max - 7 + e, so
// that weights times scales stay below 2^7 and the fp16 they are rounded to is
// far from both of its ends.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "attend_device.cuh"
#include "device_common.cuh"

namespace w12 {

namespace {

constexpr int kGW = 4;                  // warps of a worker
constexpr int kGT = kGW * 32;
constexpr int kCW = 2 * kGW;            // consumer warps
constexpr float kNegInf = -INFINITY;

// Bytes of the keys (or values) of a tile, and of a stage as the boxes lay
// it: keys, values, then (e4m3) 64 key scales and 64 value scales.  bf16 rows
// of 128 channels are two 128-byte halves (all rows of the first, then of
// the second).
template <int D, bool Q8, int NR>
struct ACfg {
    static constexpr int RT = 8 * NR;
    // A copy takes its issuing thread some 100 cycles, so a worker's keys,
    // values and e4m3 scales have a warp each (with one warp for all three
    // the stream stops at 4.4 TB/s): warpgroups 2 and, e4m3, 3.
    static constexpr int kThreads = Q8 ? 512 : 384;
    static constexpr int kProducers = Q8 ? 3 : 2;
    // registers: shares of the launch's 16 x 128 or 12 x 168 per lane
    static constexpr int kRegsConsumer = Q8 ? 200 : 216, kRegsProducer = Q8 ? 56 : 72;
    static_assert(8 * kRegsConsumer + (kThreads / 32 - 8) * kRegsProducer <= (Q8 ? 16 * 128 : 12 * 168), "register shares");
    static constexpr int kTileBytes = kAttTile * D * (Q8 ? 1 : 2);
    static constexpr int kScaleOff = 2 * kTileBytes;
    static constexpr int kStage = 2 * kTileBytes + (Q8 ? 1024 : 0);
    // per worker, after the rings: queries, the join's step, row statistics
    static constexpr int kQ = RT * D * 2;
    static constexpr int kJoinCols = 64;                            // channels per step of the workers' join
    static constexpr int kJoinPitch = kJoinCols + 4;
    static constexpr int kJoin = kGW * 8 * kJoinPitch * 4;
    static constexpr int kStat = kGW * RT * 8 + RT * 8 + RT * 4;    // per warp and row (m, l); (m, 1 / l); query scale
    static constexpr int kWorker = kQ + kJoin + kStat;
    static constexpr int kPlan = (int(sizeof(AttShared)) + 15) / 16 * 16;
    static constexpr int kMisc = 512;                               // barriers, wait state
    static constexpr int kFixed = 2 * kWorker + kPlan + kMisc;
    static constexpr int kFit = (227 * 1024 - kFixed) / (2 * kStage);
    static constexpr int S = kFit > 8 ? 8 : kFit;                   // stages per worker
    static constexpr size_t kSmem = size_t(2 * S) * kStage + kFixed;
    static_assert(S >= 2 && kSmem <= 227 * 1024 && 4 * S * 8 + 64 <= kMisc, "shared memory");
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

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float lds_f32(uint32_t addr) { return __uint_as_float(lds32(addr)); }

// A 16-byte piece of a value row with a channel that is not finite.
template <bool Q8>
__device__ __forceinline__ bool odd_values(const uint4 &x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (Q8)
#pragma unroll
            for (int b = 0; b < 4; ++b) bad = bad || ((w[e] >> (8 * b)) & 0x7Fu) == 0x7Fu;
        else
            bad = bad || (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
    return bad;
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Channel of row g8 (h = 0) or g8 + 8 (h = 1) of output block t (16 channels):
// the bf16 tiles are read in plain order; an e4m3 lane reads 16 (or 8)
// neighbouring channels of a value row at once, and numbers 2 t and 2 t + 1
// of them serve block t.
template <int D, bool Q8>
__device__ __forceinline__ int out_channel(int t, int h, int g8) {
    if (!Q8) return 16 * t + 8 * h + g8;
    if (D == 128) return 16 * g8 + 2 * t + h;
    return 16 * (g8 & 3) + 8 * (g8 >> 2) + 2 * t + h;
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

__device__ __forceinline__ void worker_sync(int worker) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + worker), "r"(kGT) : "memory");
}

template <int D, bool Q8, int NR>
__global__ void __launch_bounds__(Q8 ? 512 : 384, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
    using C = ACfg<D, Q8, NR>;
    constexpr int S = C::S, RT = C::RT, KS = D / 16, MB = D / 16;  // product steps over channels, output blocks
    constexpr int PPR = D / (Q8 ? 16 : 8);                        // 16-byte pieces of a cache row
    extern __shared__ __align__(1024) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // this warp's worker: consumers 0-3 and 4-7; producers in the same order
    const int me = warp < kCW ? warp / kGW : (warp - kCW) / (Q8 ? 4 : 2);
    const uint32_t ring = smem_addr(smem) + uint32_t(me * S * C::kStage);
    unsigned char *fixed = smem + size_t(2 * S) * C::kStage + me * C::kWorker;
    const uint32_t qs = smem_addr(fixed);
    float *join = reinterpret_cast<float *>(fixed + C::kQ);
    float2 *rowstat = reinterpret_cast<float2 *>(fixed + C::kQ + C::kJoin);  // [kGW][RT]
    float2 *row_ml = rowstat + kGW * RT;                                     // [RT]
    float *q_up = reinterpret_cast<float *>(row_ml + RT);                    // [RT]
    AttShared &sh = *reinterpret_cast<AttShared *>(smem + size_t(2 * S) * C::kStage + 2 * C::kWorker);
    unsigned char *misc = smem + size_t(2 * S) * C::kStage + 2 * C::kWorker + C::kPlan;
    uint64_t *full = reinterpret_cast<uint64_t *>(misc) + me * 2 * S, *empty = full + S;
    WaitCtl &ctl = *reinterpret_cast<WaitCtl *>(misc + 4 * S * 8);
    int *s_last = reinterpret_cast<int *>(&ctl + 1);  // [2]
    if (smem_addr(smem) & 1023u) {  // the swizzled boxes need 1024-byte aligned stages
        if (threadIdx.x == 0) record_error(a.err, W12_ERR_DEVICE);
        return;
    }
    if (threadIdx.x == 0) {
        uint64_t *bar = reinterpret_cast<uint64_t *>(misc);
        for (int s = 0; s < S; ++s)
            for (int g = 0; g < 2; ++g) {
                mbar_init(&bar[g * 2 * S + s], C::kProducers);
                mbar_init(&bar[g * 2 * S + S + s], kGW);
            }
        ctl.abort = 0;
        ctl.limit_ns = kWaitLimitNs;
        mbar_fence_init();
    }
    if (lane == 0 && warp >= kCW) prefetch_map(&a.mk), prefetch_map(&a.mv);
    att_start(a);
    const AttPlan plan = att_plan(a, sh, 2, me);
    const AttendLine &ln = a.line[kLineRest];
    const int t0 = plan.t0, t1 = plan.t1;
    if (warp >= kCW) {
        // ------------------------------------------------------ producers
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsProducer));
        const int part = (warp - kCW) % (Q8 ? 4 : 2);
        if (part >= C::kProducers) return;
        const int br = min(a.page, kAttTile);
        int issued = 0;
        att_producer<kAttTile>(
            a, plan, sh, sh.first[me], br,
            [&](int i) {
                const int s = i % S;
                const bool go =
                    i < S || (att_wait(&empty[s], uint32_t(i / S - 1) & 1u, &ctl, a.err) && !aborted(&ctl));
                issued += go;
                return __all_sync(0xFFFFFFFFu, go) != 0;
            },
            [&](int i, int chunks) {
                mbar_expect_tx(&full[i % S], uint32_t(chunks * br) * uint32_t(part == 2 ? 8 : Q8 ? D : 2 * D));
            },
            [&](int i, int chunk, int row) {
                const int s = i % S;
                const uint32_t st = ring + uint32_t(s) * uint32_t(C::kStage), at = uint32_t(chunk * br);
                if (part == 2) {
                    const uint32_t sc = st + uint32_t(C::kScaleOff) + at * 4u;
                    bulk_bytes(sc, a.ks + row, uint32_t(br) * 4u, &full[s]);
                    bulk_bytes(sc + kAttTile * 4u, a.vs + row, uint32_t(br) * 4u, &full[s]);
                } else {
                    const CUtensorMap *map = part ? &a.mv : &a.mk;
                    const uint32_t to = st + uint32_t(part ? C::kTileBytes : 0);
                    if (Q8) {
                        tma_box(to + at * uint32_t(D), map, 0, row, &full[s]);
                    } else {
#pragma unroll
                        for (int h = 0; h < D / 64; ++h)
                            tma_box(to + uint32_t(h * kAttTile * 128) + at * 128u, map, 64 * h, row, &full[s]);
                    }
                }
            });
        // after a timeout: let the copies in flight land before the CTA ends
        if (lane == 0 && aborted(&ctl))
            for (int j = issued - 1; j >= 0 && j >= issued - S; --j)
                mbar_drain(&full[j % S], uint32_t(j / S) & 1u, kAttDrainNs);
        return;
    }

    // ------------------------------------------------------------ consumers
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsConsumer));
    const int tid = threadIdx.x & (kGT - 1), wg = warp & (kGW - 1);
    const int kw = 16 * wg;                           // this warp's keys of a tile
    const int g8 = lane >> 2, q4 = lane & 3;
    const int r0 = lane & 7, mat = lane >> 3;         // ldmatrix: this lane's row and matrix
    if (t0 >= t1) {
        att_end(a);
        return;
    }
    AttSeg seg = sh.first[me];
    // a thread's share of a segment's query rows: 16-byte pieces tid, tid + kGT ..
    constexpr int kQP = RT * D / 8 / kGT ? RT * D / 8 / kGT : 1;
    uint4 qn[kQP];
    const auto load_q = [&](const AttSeg &s) {
#pragma unroll
        for (int x = 0; x < kQP; ++x) {
            const int row = (tid + x * kGT) / (D / 8), c = (tid + x * kGT) % (D / 8);
            qn[x] = make_uint4(0, 0, 0, 0);
            if (row < s.nrows && row < RT) {
                const int rho = s.row0 + row, tok = att_token(a, rho), hq = s.head * a.G + rho - tok * a.G;
                qn[x] = *reinterpret_cast<const uint4 *>(a.q + tok * a.q_stride + int64_t(hq) * D + 8 * c);
            }
        }
    };
    load_q(seg);
#pragma unroll 1
    for (int t = t0;;) {
        const int n_tiles = min(seg.left, t1 - t);
        // ---- query rows into shared memory (rows past the unit: zeros), and
        // the next segment's on their way
        worker_sync(me);  // the previous segment's copy is no longer read
#pragma unroll
        for (int x = 0; x < kQP; ++x) {
            const int row = (tid + x * kGT) / (D / 8), c = (tid + x * kGT) % (D / 8);
            const uint32_t w[4] = {qn[x].x, qn[x].y, qn[x].z, qn[x].w};
            if (!Q8) {
                if (row < RT)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(query_at<D>(qs, row, c)), "r"(w[0]),
                                 "r"(w[1]), "r"(w[2]), "r"(w[3])
                                 : "memory");
            } else {
                // the row's largest magnitude (the D / 8 lanes of a row are neighbours)
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
                top = __reduce_max_sync(D == 128 ? 0xFFFFu << (lane & 16) : 0xFFu << (lane & 24), top);
                // 2^-e with e the exponent of the largest (kept in [-100, 126])
                const int e = max(-100, min(126, int(top >> 7) - 127));
                const float down = __uint_as_float(uint32_t(127 - e) << 23);
                if (row < RT) {
                    if (c == 0) q_up[row] = __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t p = pack_f16(bf16_bits_to_float(w[j] & 0xFFFFu) * down,
                                                    bf16_bits_to_float(w[j] >> 16) * down);
                        const int col = query_column<Q8>(8 * c + 2 * j);
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(query_at<D>(qs, row, col >> 3) + uint32_t(col & 7) * 2u),
                                     "r"(p)
                                     : "memory");
                    }
                }
            }
        }
        AttSeg next = seg;
        const bool more = t + n_tiles < t1;
        if (more) {
            att_next(a, plan, sh, next);
            load_q(next);
        }
        worker_sync(me);
        // a lane has query rows 8 n + 2 q4 + c, n < NR, c < 2
        float up[NR][2];  // scale in log2 units (times the query row's power of two)
        int pos[NR][2];
        int min_pos = 0x7FFFFFFF;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 8 * n + 2 * q4 + c;
                up[n][c] = a.scale_log2 * (Q8 ? q_up[row] : 1.0f);
                pos[n][c] = 0x7FFFFFFF;  // rows past the unit: their results are not kept
                if (row < seg.nrows)  // (a unit's rows are of one request)
                    pos[n][c] = seg.key_end - a.T + att_token(a, seg.row0 + row) - seg.req * a.T;
                min_pos = min(min_pos, pos[n][c]);
            }
        min_pos = __reduce_min_sync(0xFFFFFFFFu, min_pos);
        uint32_t qf[NR][KS][2];
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int ks = 0; ks < KS; ks += 2) {
                uint32_t x[4];
                ldsm4(x, query_at<D>(qs, 8 * n + r0, 2 * ks + mat));
                qf[n][ks][0] = x[0], qf[n][ks][1] = x[1];
                qf[n][ks + 1][0] = x[2], qf[n][ks + 1][1] = x[3];
            }

        float o[MB][NR][4];
        float m_run[NR][2], l_run[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            m_run[n][0] = m_run[n][1] = kNegInf;
            l_run[n][0] = l_run[n][1] = 0.0f;
#pragma unroll
            for (int b = 0; b < MB; ++b) o[b][n][0] = o[b][n][1] = o[b][n][2] = o[b][n][3] = 0.0f;
        }

#pragma unroll 1
        for (int k = 0; k < n_tiles; ++k) {
            const int i = t - t0 + k, s = i % S;
            att_wait(&full[s], uint32_t(i / S) & 1u, &ctl, a.err);
            const uint32_t kb = ring + uint32_t(s) * uint32_t(C::kStage), vb = kb + uint32_t(C::kTileBytes);
            const int key0 = seg.key + k * kAttTile + kw;  // this warp's first key
            const bool whole = key0 + 16 <= seg.key_end && key0 + 15 <= min_pos;

            // ---- scores of 16 keys: sc[n][2 h + c], key g8 + 8 h; one block
            // of rows: in two chains
            float sc[NR][4], sc2[NR == 1 ? 1 : NR][4];
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) sc[n][x] = sc2[n][x] = 0.0f;
            uint4 kx[2][Q8 ? D / 64 : 1];  // e4m3: a lane's pieces q4 (and q4 + 4) of keys g8 and g8 + 8
            if (Q8)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int p = 0; p < D / 64; ++p)
                        kx[h][Q8 ? p : 0] = lds128(tile_at<D, Q8>(kb, kw + 8 * h + g8, q4 + 4 * p));
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t kf[4];
                if (Q8) {
                    uint32_t w[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 &x = kx[h][Q8 ? ks >> 2 : 0];
                        w[h] = (ks & 3) == 0 ? x.x : (ks & 3) == 1 ? x.y : (ks & 3) == 2 ? x.z : x.w;
                    }
                    kf[0] = e4m3x2_lo_to_f16x2(w[0]), kf[1] = e4m3x2_lo_to_f16x2(w[1]);
                    kf[2] = e4m3x2_hi_to_f16x2(w[0]), kf[3] = e4m3x2_hi_to_f16x2(w[1]);
                } else {
                    ldsm4(kf, tile_at<D, Q8>(kb, kw + 8 * (mat & 1) + r0, 2 * ks + (mat >> 1)));
                }
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    mma16816<Q8>(NR == 1 && (ks & 1) ? sc2[0] : sc[n], kf, qf[n][ks][0], qf[n][ks][1]);
            }
            if (NR == 1)
#pragma unroll
                for (int x = 0; x < 4; ++x) sc[0][x] += sc2[0][x];
            // ---- values: on their way during the softmax, but for a tile
            // whose value rows are changed below
            constexpr int W = Q8 ? (D == 128 ? 4 : 2) : 1;  // e4m3: words of a lane's piece of a value row
            uint32_t vx[4][W], vf[Q8 ? 1 : MB][4];
            const auto load_v = [&] {
                if (Q8) {
                    const int ka = kw + 2 * q4;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key = ka + (j & 1) + 8 * (j >> 1);
                        if (D == 128) {
                            const uint4 x = lds128(tile_at<D, Q8>(vb, key, g8));
                            vx[j][0] = x.x, vx[j][W > 1 ? 1 : 0] = x.y, vx[j][W > 2 ? 2 : 0] = x.z, vx[j][W > 3 ? 3 : 0] = x.w;
                        } else {
                            const uint2 x = lds64(tile_at<D, Q8>(vb, key, g8 & 3) + 8u * uint32_t(g8 >> 2));
                            vx[j][0] = x.x, vx[j][W > 1 ? 1 : 0] = x.y;
                        }
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < MB; ++b)
                        ldsm4t(vf[Q8 ? 0 : b], tile_at<D, Q8>(vb, kw + r0 + 8 * (mat >> 1), 2 * b + (mat & 1)));
                }
            };
            float kscale[2] = {1.0f, 1.0f}, vscale[2] = {1.0f, 1.0f};
            float lift[NR][2];  // e4m3: e - 7 for value scales below 2^e
#pragma unroll
            for (int n = 0; n < NR; ++n) lift[n][0] = lift[n][1] = 0.0f;
            if (Q8) {
                const uint32_t sb = kb + uint32_t(C::kScaleOff) + uint32_t(kw + g8) * 4u;
                uint32_t top = 0u;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    kscale[h] = lds_f32(sb + 32u * uint32_t(h));
                    vscale[h] = lds_f32(sb + kAttTile * 4u + 32u * uint32_t(h));
                    // scales of rows that are not the unit's may be anything
                    if (key0 + 8 * h + g8 >= seg.key_end) kscale[h] = vscale[h] = 0.0f;
                    // (a NaN scale makes the rows that see the key NaN by itself)
                    if (vscale[h] <= 3.0e38f) top = max(top, __float_as_uint(vscale[h]));
                }
                const float all = exp_above(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, top))) - 7.0f;
#pragma unroll
                for (int n = 0; n < NR; ++n) lift[n][0] = lift[n][1] = all;
            }
            if (whole) {
                load_v();
            } else if (Q8 && min(key0 + 15, seg.key_end - 1) > min_pos) {
                // keys that some row does not see: each row's bound is of the
                // scales that it sees (the same, as a rule, for all rows)
                float common = 0.0f, top[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    top[h] = vscale[h] <= 3.0e38f ? vscale[h] : 0.0f;
                    if (key0 + 8 * h + g8 <= min_pos) common = fmaxf(common, top[h]);
                }
                common = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(common)));
                if (exp_above(common) - 7.0f != lift[0][0]) {
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float x = fmaxf(key0 + g8 <= pos[n][c] ? top[0] : 0.0f, key0 + 8 + g8 <= pos[n][c] ? top[1] : 0.0f);
#pragma unroll
                            for (int off = 4; off <= 16; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, off));
                            lift[n][c] = exp_above(x) - 7.0f;
                        }
                }
            }
            // ---- mask, running maximum, weights
            float pw[NR][4];
            uint32_t pf[NR][2];
            bool moved = false;
            float alpha[NR][2];
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                float x[2][2], mx[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        x[c][h] = sc[n][2 * h + c] * up[n][c];
                        if (Q8) x[c][h] *= kscale[h];
                        const int j = key0 + 8 * h + g8;
                        if (!whole && (j >= seg.key_end || j > pos[n][c])) x[c][h] = kNegInf;
                    }
                    mx[c] = fmaxf(x[c][0], x[c][1]);
                }
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1)
#pragma unroll
                    for (int c = 0; c < 2; ++c) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xFFFFFFFFu, mx[c], off));
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float mn = fmaxf(m_run[n][c], mx[c] + lift[n][c]);
                    const float mu = mn == kNegInf ? 0.0f : mn;  // a row without keys so far
                    alpha[n][c] = ex2(m_run[n][c] - mu);
                    moved = moved || m_run[n][c] != mn;
                    m_run[n][c] = mn;
                    const float p0 = ex2(x[c][0] - mu), p1 = ex2(x[c][1] - mu);
                    l_run[n][c] = l_run[n][c] * alpha[n][c] + (p0 + p1);
                    // a masked weight is zero whatever the key's scale holds
                    pw[n][c] = !Q8 ? p0 : p0 == 0.0f ? 0.0f : p0 * vscale[0];
                    pw[n][2 + c] = !Q8 ? p1 : p1 == 0.0f ? 0.0f : p1 * vscale[1];
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    pf[n][h] = transpose8x8(Q8 ? pack_f16(pw[n][2 * h], pw[n][2 * h + 1])
                                               : pack_bf16(pw[n][2 * h], pw[n][2 * h + 1]));
            }
            if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[b][n][x] *= alpha[n][x & 1];
            }
            // ---- value rows that some query row must not see
            if (!whole) {
                bool touched = false, bad = false;
                // rows past the unit's keys (another request's, or never
                // written) are taken as zeros: 0 * NaN would reach the sum;
                // keys that only some rows see are looked at for channels
                // that are not finite
#pragma unroll 2
                for (int x = lane; x < 16 * PPR; x += 32) {
                    const int kr = x / PPR, c = x % PPR;
                    const uint32_t at = tile_at<D, Q8>(vb, kw + kr, c);
                    if (key0 + kr >= seg.key_end) {
                        sts_zero16(at);
                        touched = true;
                    } else if (key0 + kr > min_pos) {
                        bad = bad || odd_values<Q8>(lds128(at));
                    }
                }
                if (__any_sync(0xFFFFFFFFu, bad)) {
                    // a row of values with such a channel is kept out of the
                    // matrix product and added to the rows that see it by itself
#pragma unroll 1
                    for (int kr = 0; kr < 16; ++kr) {
                        const int j = key0 + kr;
                        if (j >= seg.key_end || j <= min_pos) continue;
                        if (!__any_sync(0xFFFFFFFFu, lane < PPR && odd_values<Q8>(lds128(tile_at<D, Q8>(vb, kw + kr, lane % PPR)))))
                            continue;
                        const int src = 4 * (kr & 7) + q4;  // the lane that has this key's weights of my rows
#pragma unroll
                        for (int n = 0; n < NR; ++n)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const float p = __shfl_sync(0xFFFFFFFFu, kr >= 8 ? pw[n][2 + c] : pw[n][c], src);
                                if (j <= pos[n][c]) {
#pragma unroll
                                    for (int b = 0; b < MB; ++b)
#pragma unroll
                                        for (int h = 0; h < 2; ++h) {
                                            const int d = out_channel<D, Q8>(b, h, g8);
                                            float v;
                                            if (Q8) {
                                                float f[4];
                                                e4m3x4_to_float(
                                                    lds_u8(tile_at<D, Q8>(vb, kw + kr, d >> 4) + uint32_t(d & 15)), f);
                                                v = f[0];
                                            } else {
                                                v = bf16_bits_to_float(
                                                    lds_u16(tile_at<D, Q8>(vb, kw + kr, d >> 3) + uint32_t(d & 7) * 2u));
                                            }
                                            o[b][n][2 * h + c] += p * v;
                                        }
                                }
                            }
                        __syncwarp();
                        if (lane < PPR) sts_zero16(tile_at<D, Q8>(vb, kw + kr, lane));
                        touched = true;
                        __syncwarp();
                    }
                }
                if (touched) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next box lands here
                __syncwarp();
            }
            if (!whole) load_v();
            // ---- weights times values
            if (Q8) {
#pragma unroll
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // channels 4 w + 2 e and the next, of keys (2 q4, 2 q4 + 1) and 8 later
                        const uint32_t sel = e ? 0x7362u : 0x5140u;
                        const uint32_t x = prmt2(vx[0][w], vx[1][w], sel), y = prmt2(vx[2][w], vx[3][w], sel);
                        const uint32_t f[4] = {e4m3x2_lo_to_f16x2(x), e4m3x2_hi_to_f16x2(x), e4m3x2_lo_to_f16x2(y),
                                               e4m3x2_hi_to_f16x2(y)};
#pragma unroll
                        for (int n = 0; n < NR; ++n) mma16816<true>(o[2 * w + e][n], f, pf[n][0], pf[n][1]);
                    }
            } else {
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int n = 0; n < NR; ++n) mma16816<false>(o[b][n], vf[Q8 ? 0 : b], pf[n][0], pf[n][1]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }

        // ---- the segment's end: add up the worker's four (m, l, O) in warp order
        int first, n_seg;
        att_unit_segments(a, plan, sh, seg, first, n_seg);
        const bool alone = n_seg == 1 && !a.join;  // the only result of its rows
        const int64_t entry = int64_t(seg.unit) + 2 * int(blockIdx.x) + me;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = l_run[n][c];
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
                if (g8 == 0) rowstat[wg * RT + 8 * n + 2 * q4 + c] = make_float2(m_run[n][c], l);
            }
        worker_sync(me);
        if (tid < RT) {
            const int row = tid;
            float m = kNegInf;
#pragma unroll
            for (int w = 0; w < kGW; ++w) m = fmaxf(m, rowstat[w * RT + row].x);
            const float mu = m == kNegInf ? 0.0f : m;
            float l = 0.0f;
#pragma unroll
            for (int w = 0; w < kGW; ++w) l += rowstat[w * RT + row].y * ex2(rowstat[w * RT + row].x - mu);
            row_ml[row] = make_float2(mu, l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l));  // no key: zeros
            if (row < seg.nrows) {
                if (alone)
                    att_store_lse(a, seg.head, seg.row0 + row, mu, l);
                else
                    ln.part_ml[entry * RT + row] = make_float2(m, l);
            }
        }
        worker_sync(me);
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float f[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) f[c] = ex2(m_run[n][c] - row_ml[8 * n + 2 * q4 + c].x);
#pragma unroll
            for (int b0 = 0; b0 < MB; b0 += C::kJoinCols / 16) {
                // kJoinCols channels of 8 rows per step; column 16 b + 8 h + g8
                // is out_channel(b0 + b, h, g8)
#pragma unroll
                for (int b = 0; b < C::kJoinCols / 16; ++b)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        join[(wg * 8 + 2 * q4 + (x & 1)) * C::kJoinPitch + 16 * b + 8 * (x >> 1) + g8] =
                            o[b0 + b][n][x] * f[x & 1];
                worker_sync(me);
                // a thread: two neighbouring channels d, d + 1 of a row
#pragma unroll
                for (int y = tid; y < 4 * C::kJoinCols; y += kGT) {
                    const int jr = y & 7, pi = y >> 3, row = 8 * n + jr;
                    const int c0 = Q8 ? 16 * (pi >> 3) + (pi & 7) : 2 * pi, c1 = c0 + (Q8 ? 8 : 1);
                    const int d = Q8 ? out_channel<D, Q8>(b0 + (pi >> 3), 0, pi & 7) : 16 * b0 + c0;
                    float x0 = 0.0f, x1 = 0.0f;
#pragma unroll
                    for (int w = 0; w < kGW; ++w) {
                        x0 += join[(w * 8 + jr) * C::kJoinPitch + c0];
                        x1 += join[(w * 8 + jr) * C::kJoinPitch + c1];
                    }
                    if (row < seg.nrows) {
                        if (alone) {
                            const float inv = row_ml[row].y;
                            *reinterpret_cast<uint32_t *>(att_out<D>(a, seg.head, seg.row0 + row) + d) =
                                pack_bf16(x0 * inv, x1 * inv);
                        } else {
                            *reinterpret_cast<float2 *>(&ln.part_o[(entry * RT + row) * D + d]) = make_float2(x0, x1);
                        }
                    }
                }
                worker_sync(me);
            }
        }
        if (!alone && !a.join) {
            // the worker that is done with the unit's last segment adds them up
            if (tid == 0) s_last[me] = att_last(a, first, n_seg);  // (the step above ended with a barrier)
            worker_sync(me);
            if (s_last[me]) {
                // (short code: the worker runs it once, and its SM has not
                // met it before; with a load per channel and entry, or in
                // 300 instructions, this took 9 or 6 us for 9 entries)
                constexpr int L = D / 8;  // lanes per row, 8 channels each
                const int d0 = tid % L * 8;
#pragma unroll 1
                for (int row = tid / L; row < seg.nrows; row += kGT / L) {
                    float m = kNegInf, l = 0.0f, acc[8] = {};
                    const size_t at = (size_t(seg.unit) + first) * RT + row;
                    att_add<D, true, 8, 8>(ln.part_ml + at, ln.part_o + at * D + d0, RT, n_seg, m, l, acc);
                    const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
                    uint2 *dst = reinterpret_cast<uint2 *>(att_out<D>(a, seg.head, seg.row0 + row) + d0);
#pragma unroll
                    for (int c = 0; c < 8; c += 4)
                        dst[c / 4] = make_uint2(pack_bf16(acc[c] * inv, acc[c + 1] * inv),
                                                pack_bf16(acc[c + 2] * inv, acc[c + 3] * inv));
                    if (d0 == 0) att_store_lse(a, seg.head, seg.row0 + row, m == kNegInf ? 0.0f : m, l);
                }
            }
        }
        if (!more) break;
        t += n_tiles;
        seg = next;
    }
    att_end(a);
}

// The join of the lines' results.  `split` warps of a block share 32 query
// rows of a head (a lane each) and kJC channels: they take parts of the
// entries, which are then added up in their order.
constexpr int kJC = 4;

template <int D, bool SPLIT>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = (a.rows + 31) / 32, slices = D / kJC, sp = SPLIT ? a.split : 1, mine = SPLIT ? warp % sp : 0;
    const int w = (int(blockIdx.x) * 8 + warp) / sp;
    pdl_launch_dependents();
    pdl_wait_previous();
    const int d0 = w % slices * kJC, head = w / slices / groups;
    const int rho = w / slices % groups * 32 + lane;
    const bool valid = head < a.heads && rho < a.rows;
    float m = kNegInf, l = 0.0f, acc[kJC] = {};
    if (valid) {
        const int tg = a.T * a.G, r = rho / tg, in_req = rho - r * tg;
        const AttendLine &lp = a.line[kLinePrefix], &lq = a.line[a.line[kLineRequests].grid ? kLineRequests : kLineRest];
        const int32_t *cum = a.plan + 3;
        const int np = a.plan[0], gp = a.plan[1], gq = a.plan[2], q0 = cum[r], q1 = cum[r + 1], qa = cum[a.R];
        int c, n;
        const int s = in_req / lq.rt;
        att_segments(gq, a.heads * lq.su * qa, head * lq.su * qa + lq.su * q0 + s * (q1 - q0), q1 - q0, c, n);
        const int u = (head * a.R + r) * lq.su + s;
        n *= lq.halves;
        int e0 = n * mine / sp, e1 = n * (mine + 1) / sp;
        if (a.line[kLineRequests].grid) {
            const size_t at = (size_t(u + c) * lq.halves + e0) * lq.rt, r0 = in_req - s * lq.rt;
            att_add<D, false, kJC, 4>(lq.part_ml + at + r0, lq.part_o + at * D + d0 * lq.rt + r0, lq.rt, e1 - e0, m, l, acc);
        } else {
            const size_t at = size_t(u + c + e0) * lq.rt + in_req;
            att_add<D, true, kJC, 2>(lq.part_ml + at, lq.part_o + at * D + d0, lq.rt, e1 - e0, m, l, acc);
        }
        if (np > 0 && att_len(a, a.kv_len[r]) > 0) {  // (a request without keys has no prefix either)
            const int b = rho / lp.rt, up = head * lp.pu + b;
            att_segments(gp, a.heads * lp.pu * np, up * np, np, c, n);
            n *= lp.halves;
            e0 = n * mine / sp, e1 = n * (mine + 1) / sp;
            const size_t at = (size_t(up + c) * lp.halves + e0) * lp.rt, r0 = rho - b * lp.rt;
            att_add<D, false, kJC, 4>(lp.part_ml + at + r0, lp.part_o + at * D + d0 * lp.rt + r0, lp.rt, e1 - e0, m, l, acc);
        }
    }
    if (SPLIT) {
        __shared__ float part[8][32][kJC + 2];
        float *o = part[warp][lane];
        o[0] = m, o[1] = l;
#pragma unroll
        for (int c = 0; c < kJC; ++c) o[2 + c] = acc[c];
        __syncthreads();
        if (mine) return;
        float top = m;
        for (int k = 1; k < sp; ++k) top = fmaxf(top, part[warp + k][lane][0]);
        const float mu = top == kNegInf ? 0.0f : top;
        float f = ex2(m - mu);
        l *= f;
#pragma unroll
        for (int c = 0; c < kJC; ++c) acc[c] *= f;
        for (int k = 1; k < sp; ++k) {
            const float *y = part[warp + k][lane];
            f = ex2(y[0] - mu);
            l += y[1] * f;
#pragma unroll
            for (int c = 0; c < kJC; ++c) acc[c] += y[2 + c] * f;
        }
        m = top;
    }
    if (!valid) return;
    const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);  // no key: zeros
    *reinterpret_cast<uint2 *>(att_out<D>(a, head, rho) + d0) =
        make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    if (d0 == 0) att_store_lse(a, head, rho, m == kNegInf ? 0.0f : m, l);
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
template <int D, bool Q8, int NR>
int run(const AttendArgs &a, void *stream) {
    using C = ACfg<D, Q8, NR>;
    static std::atomic<uint64_t> ready[4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return W12_ERR_CUDA;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(ready[dev >> 6].load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(attend_kernel<D, Q8, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(C::kSmem)) != cudaSuccess)
            return W12_ERR_CUDA;
        ready[dev >> 6].fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_step(attend_kernel<D, Q8, NR>, a.line[kLineRest].grid / 2, C::kThreads, C::kSmem, 1, stream, a);
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

template <int D, bool Q8>
int run_rows(const AttendArgs &a, void *stream) {
    const int rt = a.line[kLineRest].rt;
    return rt == 8 ? run<D, Q8, 1>(a, stream) : run<D, Q8, 2>(a, stream);
}

int launch_attend_rest(const AttendArgs &a, int dim, int kv, void *stream) {
    const bool q8 = kv == W12_KV_E4M3;
    if (dim == 128) return q8 ? run_rows<128, true>(a, stream) : run_rows<128, false>(a, stream);
    return q8 ? run_rows<64, true>(a, stream) : run_rows<64, false>(a, stream);
}

int launch_attend_join(const AttendArgs &a, int dim, void *stream) {
    const int64_t warps = int64_t((a.rows + 31) / 32) * a.heads * (dim / kJC) * a.split;
    const int blocks = int((warps + 7) / 8);
    if (a.split > 1)
        return dim == 128 ? launch_step(attend_join_kernel<128, true>, blocks, 256, 0, 1, stream, a)
                          : launch_step(attend_join_kernel<64, true>, blocks, 256, 0, 1, stream, a);
    return dim == 128 ? launch_step(attend_join_kernel<128, false>, blocks, 256, 0, 1, stream, a)
                      : launch_step(attend_join_kernel<64, false>, blocks, 256, 0, 1, stream, a);
}

}  // namespace w12
