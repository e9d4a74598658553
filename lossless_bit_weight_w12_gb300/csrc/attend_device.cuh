// attend_device.cuh -- the work split of attention over the paged cache, and
// what its kernels share.
//
// Query rows of one key head: row rho = token * G + g, token = request * T +
// i, G = query heads per key head; a request's rows are consecutive.  Keys
// come in tiles of kAttTile on one grid.  A unit is a block of rt query rows
// of one head against one stretch of keys:
//  - prefix unit p < pu: rows [p rt, (p + 1) rt) of ALL requests against the
//    keys [0, prefix), read once through request 0's table;
//  - request unit (r, s), s < su: rows s rt .. of request r against its own
//    keys [prefix, kv_len[r]).
// Up to three launches ("lines") share the tiles.  Where a part has enough
// rows, its whole tiles (every key of the tile seen by every row) go to the
// tensor-memory kernel, which then needs no masks; what is left -- the tile
// that the prefix ends in, the tiles of the draft block and of a ragged end,
// parts with few rows -- goes to the register kernel.
// Within a line, units of a head are ordered prefix first, then by r and s;
// heads in order.  All tiles of all units form one row, cut into equal
// pieces, one per CTA: every CTA streams the same number of tiles whatever
// the lengths are.  A CTA's share of a unit is a segment; it leaves its
// (m, l, O) -- reference exponent, sum and unnormalised output -- in slot
// (unit + CTA), which no other segment has: from one segment to the next
// either the unit or the CTA goes up, never down.  The join kernel adds up
// each row's segments in a fixed order, so results do not depend on timing.
#pragma once

#include "async_common.cuh"
#include "step_device.cuh"
#include "step_internal.h"

namespace w12 {

constexpr int kAttMaxR = W12_ATTEND_MAX_R;

// Shared memory of the plan that every CTA makes for itself.
struct AttShared {
    int lens[kAttMaxR];
    int cum[kAttMaxR + 1];  // tiles of the requests before r, one row block each
    int shortest, longest;
};

struct AttSeg {
    int head, unit;         // unit: global index
    int req;                // table row
    int row0, nrows;        // query rows
    int tile, left;         // key tile, tiles of the unit from here on
    int skip_at, skip;      // after skip_at tiles the unit goes on `skip` tiles later
    int key_begin, key_end;
    __device__ __forceinline__ int key(int k) const { return (tile + k + (k >= skip_at ? skip : 0)) * kAttTile; }
};

__device__ __forceinline__ int att_len(const AttendArgs &a, int n) {
    const int64_t room = a.table_cols << a.page_log2;
    const int cap = room < a.max_len ? int(room) : a.max_len;
    return n < 0 ? 0 : n > cap ? cap : n;
}

// Whole tiles of the prefix (the tensor-memory kernel's), and the end of the
// prefix's keys.
__device__ __forceinline__ int att_prefix_whole(const AttendArgs &a, int shortest) {
    return a.line[kLinePrefix].grid ? min(a.prefix, max(shortest - a.T + 1, 0)) / kAttTile : 0;
}
__device__ __forceinline__ int att_prefix_end(const AttendArgs &a, int longest) { return min(a.prefix, longest); }

// The tensor-memory kernel's tiles [c0, c1) of a request of len keys.
__device__ __forceinline__ void att_req_whole(const AttendArgs &a, int len, int *c0, int *c1) {
    *c0 = (a.prefix + kAttTile - 1) / kAttTile;
    *c1 = a.line[kLineRequests].grid ? max(*c0, max(len - a.T + 1, 0) / kAttTile) : *c0;
}

// This line's tiles of a prefix unit and of a request.
__device__ __forceinline__ int att_prefix_tiles(const AttendArgs &a, int shortest, int longest) {
    if (!a.line[a.self].pu) return 0;
    const int w = att_prefix_whole(a, shortest);
    return a.self == kLineRest ? (att_prefix_end(a, longest) + kAttTile - 1) / kAttTile - w : w;
}
__device__ __forceinline__ int att_req_tiles(const AttendArgs &a, int len) {
    if (!a.line[a.self].su) return 0;
    int c0, c1;
    att_req_whole(a, len, &c0, &c1);
    if (a.self != kLineRest) return c1 - c0;
    return len > a.prefix ? (len + kAttTile - 1) / kAttTile - a.prefix / kAttTile - (c1 - c0) : 0;
}

// CTA c's tiles begin at att_begin(total, grid, c); the CTA that has tile t.
__device__ __forceinline__ int att_begin(int total, int grid, int c) {
    const int per = total / grid, rem = total % grid;
    return c * per + min(c, rem);
}
__device__ __forceinline__ int att_owner(int total, int grid, int t) {
    const int per = total / grid, rem = total % grid;
    return t < rem * (per + 1) ? t / (per + 1) : rem + (t - rem * (per + 1)) / per;
}

struct AttPlan {
    int np;        // tiles of a prefix unit
    int per_head;  // tiles of a head
    int t0, t1;    // this CTA's tiles
};

// Lengths and cumulative tile counts into shared memory (all threads of the
// CTA); CTA 0 also leaves them for the join kernel.
__device__ __forceinline__ AttPlan att_plan(const AttendArgs &a, AttShared &sh, int threads) {
    const int lane = threadIdx.x & 31;
    const AttendLine &ln = a.line[a.self];
    for (int r = threadIdx.x; r < a.R; r += threads) {
        const int n0 = a.kv_len[r], n = att_len(a, n0);
        if (n0 > n && blockIdx.x == 0) atomicCAS(a.err, 0, W12_ERR_DEVICE);
        sh.lens[r] = n;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int sum = 0, longest = 0, shortest = 0x7FFFFFFF;
        for (int r0 = 0; r0 < a.R; r0 += 32) {
            const int r = r0 + lane;
            int x = 0;
            if (r < a.R) {
                const int n = sh.lens[r];
                longest = max(longest, n);
                shortest = min(shortest, n);
                x = att_req_tiles(a, n);
            }
            const int y = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int z = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += z;
            }
            if (r < a.R) sh.cum[r] = sum + x - y;
            sum += __shfl_sync(0xFFFFFFFFu, x, 31);
        }
        longest = __reduce_max_sync(0xFFFFFFFFu, longest);
        shortest = __reduce_min_sync(0xFFFFFFFFu, shortest);
        if (lane == 0) {
            sh.cum[a.R] = sum;
            sh.longest = longest;
            sh.shortest = shortest;
        }
    }
    __syncthreads();
    AttPlan p;
    p.np = att_prefix_tiles(a, sh.shortest, sh.longest);
    p.per_head = ln.pu * p.np + ln.su * sh.cum[a.R];
    const int total = p.per_head * a.heads;
    p.t0 = att_begin(total, ln.grid, int(blockIdx.x));
    p.t1 = att_begin(total, ln.grid, int(blockIdx.x) + 1);
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) ln.plan[0] = p.np;
        for (int r = threadIdx.x; r <= a.R; r += threads) ln.plan[1 + r] = sh.cum[r];
    }
    return p;
}

// The unit and key tile of tile t of the line.
__device__ __forceinline__ AttSeg att_locate(const AttendArgs &a, const AttPlan &p, const AttShared &sh, int t) {
    const AttendLine &ln = a.line[a.self];
    AttSeg s;
    s.head = t / p.per_head;
    s.skip_at = 0x7FFFFFFF;
    s.skip = 0;
    int w = t - s.head * p.per_head;
    const int units = ln.pu + a.R * ln.su;
    if (w < ln.pu * p.np) {
        const int u = w / p.np;
        s.unit = s.head * units + u;
        s.req = 0;
        s.row0 = u * ln.rt;
        s.nrows = min(ln.rt, a.rows - s.row0);
        s.left = p.np - (w - u * p.np);
        s.tile = (a.self == kLineRest ? att_prefix_whole(a, sh.shortest) : 0) + (w - u * p.np);
        s.key_begin = 0;
        s.key_end = att_prefix_end(a, sh.longest);
        return s;
    }
    w -= ln.pu * p.np;
    int lo = 0, hi = a.R;  // the last request r with cum[r] <= w / su
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.cum[mid] <= w / ln.su) lo = mid; else hi = mid;
    }
    const int r = lo, n = sh.cum[r + 1] - sh.cum[r];
    w -= sh.cum[r] * ln.su;
    const int u = w / n, k = w - u * n, tg = a.T * a.G;
    s.unit = s.head * units + ln.pu + r * ln.su + u;
    s.req = r;
    s.row0 = r * tg + u * ln.rt;
    s.nrows = min(ln.rt, tg - u * ln.rt);
    s.left = n - k;
    int c0, c1;
    att_req_whole(a, sh.lens[r], &c0, &c1);
    if (a.self == kLineRest) {
        const int first = a.prefix / kAttTile, head = c1 > c0 ? c0 - first : 0x3FFFFFFF;  // tiles before the gap
        s.tile = k < head ? first + k : c1 + (k - head);
        if (k < head && c1 > c0) s.skip_at = head - k, s.skip = c1 - c0;
    } else {
        s.tile = c0 + k;
    }
    s.key_begin = a.prefix;
    s.key_end = sh.lens[r];
    return s;
}

// ---- copies into a ring stage

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void bulk_bytes(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// Bytes of the keys (or values) of a tile, and of a stage as the boxes lay
// it: keys, values, then (e4m3) 64 key scales and 64 value scales.  bf16 rows
// of 128 channels are two 128-byte halves (all rows of the first, then of
// the second); all with the 128-byte swizzle but the 64-byte rows of e4m3
// with 64 channels (64-byte swizzle).
template <int D, bool Q8>
struct AttStage {
    static constexpr int kTile = kAttTile * D * (Q8 ? 1 : 2);
    static constexpr int kScale = 2 * kTile;
    static constexpr int kBytes = 2 * kTile + (Q8 ? 1024 : 0);
};

// The producer warp: tiles [t0, t1) of the line into a ring of S stages,
// tile i into stage i % S once `empty` says that its last tile is done with.
// A lane per box row block ("chunk": the keys of one page in one tile); a
// batch of 32 chunks has its table entries read at once, the next batch's
// while this one is issued.  full[s] is armed with the bytes of the chunks
// that hold keys of the unit.
template <int D, bool Q8, int S>
__device__ __forceinline__ void att_producer(const AttendArgs &a, const AttPlan &plan, const AttShared &sh, uint32_t ring,
                                             uint64_t *full, uint64_t *empty, WaitCtl *ctl) {
    using St = AttStage<D, Q8>;
    const int lane = threadIdx.x & 31;
    const int br = min(a.page, kAttTile), cpt = kAttTile / br, tpb = 32 / cpt;
    const int my_tile = lane / cpt, my_chunk = lane % cpt;
    struct Chunk {
        int row, valid;  // first cache row; 0: nothing to load
    };
    const auto look = [&](int tb) {
        Chunk c{0, 0};
        const int t = tb + my_tile;
        if (t >= plan.t1) return c;
        const AttSeg g = att_locate(a, plan, sh, t);
        const int key = g.key(0) + my_chunk * br;
        // (keys before the prefix's end are not looked up in the request's own row)
        if (key >= g.key_end || key + br <= g.key_begin) return c;
        int pg = a.table[int64_t(g.req) * a.table_cols + (key >> a.page_log2)];
        if (pg < 0 || pg >= a.n_pages) {
            atomicCAS(a.err, 0, W12_ERR_DEVICE);
            pg = 0;
        }
        c.row = ((pg * a.heads + g.head) << a.page_log2) + (key & (a.page - 1));
        c.valid = 1;
        return c;
    };
    int issued = 0;
    bool stop = false;
    Chunk cur = look(plan.t0);
    for (int tb = plan.t0; tb < plan.t1 && !stop; tb += tpb) {
        const Chunk nxt = look(tb + tpb);
        for (int k = 0; k < tpb && tb + k < plan.t1; ++k) {
            const int i = tb + k - plan.t0, s = i % S;
            int go = 1;
            if (lane == 0) go = i < S || (mbar_wait(&empty[s], uint32_t(i / S - 1) & 1u, ctl, a.err) && !aborted(ctl));
            go = __shfl_sync(0xFFFFFFFFu, go, 0);
            if (!go) {
                stop = true;
                break;
            }
            const bool mine = my_tile == k && cur.valid;
            const int chunks = __popc(__ballot_sync(0xFFFFFFFFu, mine));
            const uint32_t st = ring + uint32_t(s) * uint32_t(St::kBytes);
            if (lane == 0)
                mbar_expect_tx(&full[s], uint32_t(chunks) * uint32_t(br) * uint32_t(D * (Q8 ? 2 : 4) + (Q8 ? 8 : 0)));
            __syncwarp();
            if (mine) {
                const uint32_t at = uint32_t(my_chunk * br);
                if (Q8) {
                    const uint32_t o = st + at * uint32_t(D);
                    tma_box(o, &a.mk, 0, cur.row, &full[s]);
                    tma_box(o + uint32_t(St::kTile), &a.mv, 0, cur.row, &full[s]);
                    const uint32_t sc = st + uint32_t(St::kScale) + at * 4u;
                    bulk_bytes(sc, a.ks + cur.row, uint32_t(br) * 4u, &full[s]);
                    bulk_bytes(sc + kAttTile * 4u, a.vs + cur.row, uint32_t(br) * 4u, &full[s]);
                } else {
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        const uint32_t o = st + uint32_t(h * kAttTile * 128) + at * 128u;
                        tma_box(o, &a.mk, 64 * h, cur.row, &full[s]);
                        tma_box(o + uint32_t(St::kTile), &a.mv, 64 * h, cur.row, &full[s]);
                    }
                }
            }
            ++issued;
        }
        cur = nxt;
    }
    // after a timeout: let the copies in flight land before the CTA ends
    if (lane == 0 && aborted(ctl))
        for (int j = issued - 1; j >= 0 && j >= issued - S; --j)
            mbar_drain(&full[j % S], uint32_t(j / S) & 1u, ctl->limit_ns);
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Exponent e of the power of two 2^e above x (x is taken as at least 1e-30).
__device__ __forceinline__ float exp_above(float x) {
    return float(int(__float_as_uint(fmaxf(x, 1e-30f)) >> 23) - 126);
}

}  // namespace w12
