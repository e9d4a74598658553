// attend_device.cuh -- the work split of attention over the paged cache, and
// what its kernels share.
//
// Query rows of one key head: row rho = token * G + g, token = request * T +
// i, G = query heads per key head; a request's rows are consecutive.  A unit
// is a block of rt query rows of one head against one stretch of keys:
//  - prefix unit p < pu: rows [p rt, (p + 1) rt) of ALL requests against the
//    keys of the prefix, read once through the table of the first request that
//    has keys (rows of requests without any are computed and left out later);
//  - request unit (r, s), s < su: rows s rt .. of request r against its own
//    keys.
// Up to two launches ("lines") share the keys: the prefix's first W tiles of
// 128 keys, for all requests at once, and what follows, request by request
// (so the part of the prefix past 128 W keys is read by each request through
// its own table).  The prefix and requests with many rows go to the
// tensor-memory kernel, requests with few rows to the register kernel in
// tiles of 64 keys.  The two run side by side, each on its share of the SMs.
// Within a line, units of a head are ordered by p, or by r and s; heads in
// order.  All tiles of all units form one row, cut into equal pieces, one per
// worker (a CTA; in the register kernel each half of a CTA): every worker
// streams the same number of tiles whatever the lengths are.  A worker's
// share of a unit is a segment; it leaves its (m, l, O) -- reference exponent,
// sum and unnormalised output -- in slot (unit + worker), which no other
// segment has: from one segment to the next either the unit or the worker
// goes up, never down.  Where the register kernel has all the results, the
// worker that finishes a unit's last segment adds them up.  With results of
// the tensor-memory kernel a join kernel does: 40 KB and more per unit, which
// one worker takes three times as long to fetch as a whole kernel (128
// requests under a prefix: 42 us against 13).  All sums have a fixed order:
// the outputs do not depend on timing.
#pragma once

#include "async_common.cuh"
#include "step_device.cuh"
#include "step_internal.h"

namespace w12 {

constexpr int kAttMaxR = W12_ATTEND_MAX_R;

// rho / G, by the reciprocal: 2^64 / G rounded up is too large by less than 1,
// the product over 2^64 by less than rho / 2^64.  The floor is exact where that
// is below 1 / G, the least distance to the next whole number: rho * G < 2^64.
__device__ __forceinline__ int att_token(const AttendArgs &a, int rho) {
    return a.G == 1 ? rho : int(__umul64hi(uint64_t(uint32_t(rho)), a.per_g));
}

// A position on the line: a unit, its first key from here on, its tiles left.
struct AttSeg {
    int head, req, block;  // block: of the unit's rows in its request (prefix: of all rows)
    int unit;              // global index
    int row0, nrows;       // query rows
    int key, left;
    int key_end;
};

// Shared memory of the plan that every CTA makes for itself.
struct AttShared {
    int lens[kAttMaxR];
    int cum[kAttMaxR + 1];  // tiles of the requests before r, one row block each
    int w, grid, source;
    AttSeg first[2];        // the CTA's workers' first positions
};

__device__ __forceinline__ int att_len(const AttendArgs &a, int n) {
    const int64_t room = a.table_cols << a.page_log2;
    const int cap = room < a.max_len ? int(room) : a.max_len;
    return n < 0 ? 0 : n > cap ? cap : n;
}

// W: the prefix's tiles of 128 keys that are read once for all requests;
// shortest: of the lengths above 0 (a request without keys, such as an idle
// slot of a fixed batch, does not part the prefix), or 0.
__device__ __forceinline__ int att_prefix_whole(const AttendArgs &a, int shortest) {
    return a.line[kLinePrefix].grid ? min(a.prefix, max(shortest - a.T + 1, 0)) / kAttTcTile : 0;
}
// The requests' tiles of one of len keys (at least one, so that every request
// has a result).
__device__ __forceinline__ int att_req_tiles(const AttendArgs &a, int w, int len) {
    const int kt = a.line[kLineRequests].grid ? kAttTcTile : kAttTile;
    return max((len + kt - 1) / kt - w * (kAttTcTile / kt), 1);
}

// Worker c's tiles begin at att_begin(total, grid, c); the worker that has
// tile t.
__device__ __forceinline__ int att_begin(int total, int grid, int c) {
    const int per = total / grid, rem = total % grid;
    return c * per + min(c, rem);
}
__device__ __forceinline__ int att_owner(int total, int grid, int t) {
    const int per = total / grid, rem = total % grid;
    return t < rem * (per + 1) ? t / (per + 1) : rem + (t - rem * (per + 1)) / per;
}

struct AttPlan {
    int w;         // the prefix's shared tiles
    int source;    // the request whose table they are read through
    int grid;      // workers of this line
    int np;        // tiles of a prefix unit of this line
    int per_head;  // tiles of a head
    int t0, t1;    // this worker's tiles
};

// SMs that take the prefix while the others take the requests (of both more
// than the GPU has).  The prefix's kernel is bound by its chain of products
// and exponentials, the requests' by the cache stream, so side by side they
// take less than one after the other (128 requests, 16000 + 460 keys: 51 + 54
// us apart).  An SM's time, measured, in units of 100 cycles: a prefix tile of
// 256 rows 33 (128 rows: 18) and 250 a CTA; of the requests a tile of 64 keys
// 7 in the register kernel, of 128 keys 18 or 33 in the other, a unit 40.
// (That call: 98 us; with 6 and 40 100, with 8 and 45 107.)
__device__ __forceinline__ int att_prefix_sms(const AttendArgs &a, int w, int sum) {
    const AttendLine &lp = a.line[kLinePrefix];
    const bool tc = a.line[kLineRequests].grid != 0;
    const AttendLine &lq = a.line[tc ? kLineRequests : kLineRest];
    const int sms_q = tc ? lq.grid : lq.grid / 2;
    if (lp.grid + sms_q <= a.sms) return lp.grid;
    const float tp = float(a.heads) * float(lp.pu) * float(w) * (lp.rt == 256 ? 33.0f : 18.0f);
    const float tq = float(a.heads) * (float(lq.su) * float(sum) * (tc ? lq.rt == 256 ? 33.0f : 18.0f : 7.0f) +
                                       float(a.R) * float(lq.su) * 40.0f);
    // tp / x + 250 = tq / (sms - x), by a few steps from the ratio
    float x = float(a.sms) * tp / (tp + tq);
    for (int k = 0; k < 4; ++k) x = float(a.sms) * (tp + 250.0f * x) / (tp + 250.0f * x + tq);
    return max(a.sms - sms_q, max(1, min(min(lp.grid, a.sms - 1), int(x + 0.5f))));
}

// Workers of the tensor-memory kernel: each has a few tiles (4 of 128 rows, 2
// of 256), as a segment costs about as much as two and leaves 64 KB of
// results, but no unit waits for another (4 requests x 8 tokens under one key
// head, 7500 keys: 42 us with a worker per tile, 18 so).
__device__ __forceinline__ int att_tc_grid(int grid, int rt, int units, int tiles) {
    const int few = rt == 256 ? 2 : 4;
    return min(grid, max(units, (tiles + few - 1) / few));
}

// Fills in what follows from (head, req, block) -- under the prefix from (head,
// block) -- for the unit's tile k.
__device__ __forceinline__ void att_unit_at(const AttendArgs &a, const AttPlan &p, const AttShared &sh, AttSeg &s, int k) {
    const AttendLine &ln = a.line[a.self];
    if (a.self == kLinePrefix) {
        s.req = p.source;
        s.unit = s.head * ln.pu + s.block;
        s.row0 = s.block * ln.rt;
        s.nrows = min(ln.rt, a.rows - s.row0);
        s.left = p.np - k;
        s.key = k * kAttTcTile;
        s.key_end = p.w * kAttTcTile;
        return;
    }
    const int tg = a.T * a.G;
    s.unit = (s.head * a.R + s.req) * ln.su + s.block;
    s.row0 = s.req * tg + s.block * ln.rt;
    s.nrows = min(ln.rt, tg - s.block * ln.rt);
    s.left = sh.cum[s.req + 1] - sh.cum[s.req] - k;
    s.key_end = sh.lens[s.req];
    s.key = p.w * kAttTcTile + k * (a.self == kLineRequests ? kAttTcTile : kAttTile);
}

// The last key that every row of the segment's unit sees.
__device__ __forceinline__ int att_seen_by_all(const AttendArgs &a, const AttSeg &s) {
    return a.self == kLinePrefix ? 0x7FFFFFFF : s.key_end - a.T + att_token(a, s.row0) - s.req * a.T;
}

// The position of tile t of the line.
__device__ __forceinline__ AttSeg att_locate(const AttendArgs &a, const AttPlan &p, const AttShared &sh, int t) {
    const AttendLine &ln = a.line[a.self];
    AttSeg s;
    s.head = t / p.per_head;
    int w = t - s.head * p.per_head, n = p.np;
    if (a.self != kLinePrefix) {
        int lo = 0, hi = a.R;  // the last request with cum <= w / su
        const int x = w / ln.su;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sh.cum[mid] <= x) lo = mid; else hi = mid;
        }
        s.req = lo;
        n = sh.cum[lo + 1] - sh.cum[lo];
        w -= sh.cum[lo] * ln.su;
    }
    s.block = w / n;
    att_unit_at(a, p, sh, s, w - s.block * n);
    return s;
}

// The start of the next unit that has tiles (there is one).
__device__ __forceinline__ void att_next(const AttendArgs &a, const AttPlan &p, const AttShared &sh, AttSeg &s) {
    const AttendLine &ln = a.line[a.self];
    const bool prefix = a.self == kLinePrefix;
    if (++s.block == (prefix ? ln.pu : ln.su)) {
        s.block = 0;
        do {
            if (prefix || ++s.req == a.R) s.req = 0, ++s.head;
        } while (!prefix && sh.cum[s.req + 1] == sh.cum[s.req]);
    }
    att_unit_at(a, p, sh, s, 0);
}

// Lengths and cumulative tile counts into shared memory (all threads of the
// CTA).
__device__ __forceinline__ AttPlan att_plan(const AttendArgs &a, AttShared &sh, int workers, int worker) {
    const int lane = threadIdx.x & 31;
    const AttendLine &ln = a.line[a.self];
    for (int r = threadIdx.x; r < a.R; r += int(blockDim.x)) {
        const int n0 = a.kv_len[r], n = att_len(a, n0);
        if (n0 > n && blockIdx.x == 0) atomicCAS(a.err, 0, W12_ERR_DEVICE);
        sh.lens[r] = n;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int w = 0;
        if (a.line[kLinePrefix].grid) {
            int shortest = 0x7FFFFFFF, source = 0x7FFFFFFF;
            for (int r = lane; r < a.R; r += 32)
                if (sh.lens[r] > 0) shortest = min(shortest, sh.lens[r]), source = min(source, r);
            shortest = __reduce_min_sync(0xFFFFFFFFu, shortest), source = __reduce_min_sync(0xFFFFFFFFu, source);
            w = att_prefix_whole(a, source < a.R ? shortest : 0);
            if (lane == 0) sh.source = source;
        }
        // a lane's requests are neighbours
        const int per = (a.R + 31) / 32, r0 = lane * per, r1 = min(r0 + per, a.R);
        int sum = 0;
        for (int r = r0; r < r1; ++r) sum += att_req_tiles(a, w, sh.lens[r]);
        // (the prefix's launch needs it, too, for its share of the SMs)
        int x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += z;
        }
        if (lane == 31) sh.cum[a.R] = x;
        x -= sum;
        // For the join kernel: by one CTA, the requests' part by their kernel,
        // the prefix's workers by its own (the share is float arithmetic, which
        // another compilation may round differently).
        const bool tells = a.join && blockIdx.x == 0, tell = tells && a.self != kLinePrefix;
        const bool tell_prefix = tells && a.self == kLinePrefix;
        if (lane == 31 && tell) a.plan[3 + a.R] = x + sum;
        for (int r = r0; r < r1; ++r) {
            sh.cum[r] = x;
            if (tell) a.plan[3 + r] = x;
            x += att_req_tiles(a, w, sh.lens[r]);
        }
        const int all = __shfl_sync(0xFFFFFFFFu, sh.cum[a.R], 31);
        if (lane == 0) {
            int g = ln.grid;
            if (w > 0) {
                const int gp = att_tc_grid(att_prefix_sms(a, w, all), a.line[kLinePrefix].rt,
                                           a.heads * a.line[kLinePrefix].pu, a.heads * a.line[kLinePrefix].pu * w);
                g = a.self == kLinePrefix ? gp : min(g, (a.sms - gp) * (a.line[kLineRequests].grid ? 1 : 2));
                if (tell_prefix) a.plan[1] = gp;
            }
            if (a.self == kLineRequests) g = att_tc_grid(g, ln.rt, a.heads * a.R * ln.su, a.heads * ln.su * all);
            sh.w = w;
            sh.grid = g;
            if (tell) a.plan[0] = w, a.plan[2] = g;
        }
    }
    __syncthreads();
    AttPlan p;
    p.w = sh.w;
    p.source = sh.source;  // (only looked at under a prefix)
    p.grid = sh.grid;
    p.np = a.self == kLinePrefix ? p.w : 0;
    p.per_head = a.self == kLinePrefix ? ln.pu * p.np : ln.su * sh.cum[a.R];
    const int total = p.per_head * a.heads;
    // the CTA's `workers` workers; this thread's is number `worker` of them
    const int c0 = int(blockIdx.x) * workers;
    p.t0 = att_begin(total, p.grid, min(c0 + worker, p.grid));
    p.t1 = att_begin(total, p.grid, min(c0 + worker + 1, p.grid));
    const int q = int(threadIdx.x >> 5);  // a warp finds a worker's first tile
    if (q < workers) {
        const int t = att_begin(total, p.grid, min(c0 + q, p.grid));
        if (t < total && a.self == kLinePrefix) {
            if (lane == 0) sh.first[q] = att_locate(a, p, sh, t);
        } else if (t < total) {
            const int head = t / p.per_head, at = t - head * p.per_head, x = at / ln.su;
            for (int r = lane; r < a.R; r += 32)
                if (sh.cum[r] <= x && x < sh.cum[r + 1]) {  // one lane's request
                    const int n = sh.cum[r + 1] - sh.cum[r], in_req = at - sh.cum[r] * ln.su;
                    AttSeg s;
                    s.head = head, s.req = r, s.block = in_req / n;
                    att_unit_at(a, p, sh, s, in_req - s.block * n);
                    sh.first[q] = s;
                }
        }
    }
    __syncthreads();
    return p;
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

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// The tiles' copies by a producer warp: KT keys each, a lane per box ("chunk":
// the keys of one page in one tile).  A batch of 32 chunks has its table
// entries read at once, the next batch's behind the copies of this one's
// first tile; the first batch stays in the worker's first segment, whose place
// is known.  ready(i), by all lanes: waits until the CTA's tile i may be
// written, false to stop; issue(i, chunks, chunk, row), on the lanes that have
// a chunk of it (keys chunk * br ... of the tile, cache rows row ...): copies
// it; chunks: of the tile, on its first, which arms the barrier before the
// others' copies.
template <int KT, typename Ready, typename Arm, typename Issue>
__device__ __forceinline__ void att_producer(const AttendArgs &a, const AttPlan &plan, const AttShared &sh,
                                             const AttSeg &start, int br, Ready ready, Arm arm, Issue issue) {
    const int lane = threadIdx.x & 31;
    const int cpt = KT / br, tpb = 32 / cpt;
    const int my_tile = lane / cpt, my_chunk = lane % cpt;
    struct Chunk {
        int head, key, page, chunks;  // key < 0: nothing to load; chunks: of the tile, from this one on
    };
    // (what it loads is not looked at before the batch is issued)
    const auto chunk_of = [&](int head, int req, int tile_key, int key_end) {
        Chunk c{0, -1, 0, 0};
        const int key = tile_key + my_chunk * br;
        if (key >= key_end) return c;
        c.head = head;
        c.key = key;
        c.chunks = min(cpt - my_chunk, (key_end - key + br - 1) / br);
        c.page = a.table[int64_t(req) * a.table_cols + (key >> a.page_log2)];
        return c;
    };
    if (plan.t0 >= plan.t1) return;
    Chunk cur{0, -1, 0, 0}, nxt = cur;
    int tb = plan.t0, n = min(min(tpb, start.left), plan.t1 - tb);
    if (my_tile < n) cur = chunk_of(start.head, start.req, start.key + my_tile * KT, start.key_end);
#pragma unroll 1
    for (;;) {
        int pg = cur.page;
        if (cur.key >= 0 && (pg < 0 || pg >= a.n_pages)) {
            atomicCAS(a.err, 0, W12_ERR_DEVICE);
            pg = 0;
        }
        const int row = ((pg * a.heads + cur.head) << a.page_log2) + (cur.key & (a.page - 1));
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
            const int i = tb + k - plan.t0;
            if (!ready(i)) return;
            const bool mine = my_tile == k;
            if (mine && my_chunk == 0) arm(i, cur.chunks);
            if (cpt > 1) __syncwarp();
            if (mine && cur.key >= 0) issue(i, my_chunk, row);
            if (k == 0) {
                const int t = tb + n + my_tile;
                nxt = Chunk{0, -1, 0, 0};
                if (t < plan.t1) {
                    const AttSeg g = att_locate(a, plan, sh, t);
                    nxt = chunk_of(g.head, g.req, g.key, g.key_end);
                }
            }
        }
        tb += n;
        if (tb >= plan.t1) return;
        n = min(tpb, plan.t1 - tb);
        cur = nxt;
    }
}

// After a timeout a producer lets its copies land, at most this long for each
// (a stage that another producer did not reach never completes).
constexpr uint64_t kAttDrainNs = 20000000ull;

// mbar_wait() that reads the clock only after some tries: the waits of these
// kernels are short and the clock is slow.
__device__ __forceinline__ bool att_wait(uint64_t *bar, uint32_t parity, WaitCtl *ctl, int *err) {
#pragma unroll 1
    for (int k = 0; k < 16; ++k)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity, ctl, err);
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

// Adds up n entries of a row: from pm (reference and sum) and po (channels),
// `rt` rows from entry to entry; U are in flight.  ROWS: the register kernel's
// order of the channels.
template <int D, bool ROWS, int C, int U>
__device__ __forceinline__ void att_add(const float2 *pm, const float *po, int rt, int n, float &m, float &l,
                                        float (&acc)[C]) {
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += U) {
        // (past the last entry: the last one again, with weight 0)
        float2 ml[U];
        float x[U][C];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int e = min(k0 + k, n - 1);
            ml[k] = __ldcg(pm + size_t(uint32_t(e * rt)));
            const float *src = po + size_t(uint32_t(e * rt)) * D;
            if (ROWS) {
#pragma unroll
                for (int c = 0; c < C; c += 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + c));
                    x[k][c] = v.x, x[k][c + 1] = v.y, x[k][c + 2] = v.z, x[k][c + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int c = 0; c < C; ++c) x[k][c] = __ldcg(src + c * rt);
            }
        }
        float mn = m;
#pragma unroll
        for (int k = 0; k < U; ++k) mn = fmaxf(mn, ml[k].x);
        const float mu = mn == -INFINITY ? 0.0f : mn, down = ex2(m - mu);
        m = mn;
        l *= down;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] *= down;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            // (a row without keys: the register kernel has zeros, the other anything)
            const bool none = k0 + k >= n || (!ROWS && ml[k].x == -INFINITY && ml[k].y == 0.0f);
            const float f = none ? 0.0f : ex2(ml[k].x - mu);
            l += ml[k].y * f;
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] += !ROWS && none ? 0.0f : x[k][c] * f;
        }
    }
}

// The output row of query row rho of a head, and its lse.
template <int D>
__device__ __forceinline__ uint16_t *att_out(const AttendArgs &a, int head, int rho) {
    const int tok = att_token(a, rho), hq = head * a.G + rho - tok * a.G;
    return a.out + int64_t(tok) * a.out_stride + int64_t(hq) * D;
}
__device__ __forceinline__ void att_store_lse(const AttendArgs &a, int head, int rho, float mu, float l) {
    if (!a.lse) return;
    const int tok = att_token(a, rho), hq = head * a.G + rho - tok * a.G;
    a.lse[int64_t(tok) * (a.G * a.heads) + hq] = l == 0.0f ? -INFINITY : (mu + log2f(l)) * 0.6931471805599453f;
}

// Where a unit of n tiles from b on of a line of `total` lies: its first
// worker, its segments.
__device__ __forceinline__ void att_segments(int grid, int total, int b, int n, int &first, int &segments) {
    first = att_owner(total, grid, b);
    segments = att_owner(total, grid, b + n - 1) - first + 1;
}
__device__ __forceinline__ void att_unit_segments(const AttendArgs &a, const AttPlan &p, const AttShared &sh,
                                                  const AttSeg &s, int &first, int &segments) {
    const AttendLine &ln = a.line[a.self];
    const int n = sh.cum[s.req + 1] - sh.cum[s.req];
    att_segments(p.grid, p.per_head * a.heads, s.head * p.per_head + ln.su * sh.cum[s.req] + s.block * n, n, first, segments);
}

// The kernels of a call with a prefix run side by side: the prefix's waits for
// what the stream did before and then lets the requests' start, which does not
// wait -- all that it reads was there when every CTA of the prefix's kernel had
// passed its wait -- but ends only after the prefix's kernel has ended, so that
// the join, which waits for the requests' kernel, has both's results.
__device__ __forceinline__ bool att_side_by_side(const AttendArgs &a) {
    return a.line[kLinePrefix].grid && a.self != kLinePrefix;
}
__device__ __forceinline__ void att_start(const AttendArgs &a) {
    if (a.self == kLinePrefix) pdl_wait_previous();
    pdl_launch_dependents();
    if (a.self != kLinePrefix && !att_side_by_side(a)) pdl_wait_previous();
}
__device__ __forceinline__ void att_end(const AttendArgs &a) {
    if (att_side_by_side(a)) pdl_wait_previous();
}

// True in the worker that is the last of a unit's (two or more) segments to
// get here (one thread; the others' results are behind a barrier that it has
// passed).  A worker is the first of at most one unit with several segments,
// so it names the counter.
__device__ __forceinline__ bool att_last(const AttendArgs &a, int first, int segments) {
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                 : "=r"(before)
                 : "l"(&a.arrived[first])
                 : "memory");
    const bool last = before == uint32_t(segments - 1);
    if (last) a.arrived[first] = 0u;
    return last;
}

}  // namespace w12
