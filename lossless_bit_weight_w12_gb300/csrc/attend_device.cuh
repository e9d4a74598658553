// attend_device.cuh -- the work split of attention over the paged cache.
//
// Query rows of one key head: row rho = token * G + g, token = request * T +
// i, G = query heads per key head; a request's rows are consecutive.  Keys
// come in tiles of kAttTile.  A unit is a block of rt query rows of one head
// against one stretch of keys:
//  - prefix unit p < pu: rows [p rt, (p + 1) rt) of ALL requests against the
//    keys [0, prefix), read once through request 0's table;
//  - request unit (r, s), s < su: rows s rt .. of request r against its own
//    keys [prefix, kv_len[r]) (tiles on the same grid, so the first may also
//    hold keys before prefix: masked).
// Units of a head are ordered prefix first, then by r and s; heads in order.
// All tiles of all units form one line, cut into equal pieces, one per CTA:
// every CTA streams the same number of tiles whatever the lengths are.  A
// CTA's share of a unit is a segment; it leaves the segment's running
// maximum, sum and unnormalised output in slot (unit + CTA), which no other
// segment has: from one segment to the next on the line either the unit or
// the CTA goes up, never down.  The join kernel adds up each row's segments
// in CTA order, so results do not depend on timing.
#pragma once

#include "async_common.cuh"
#include "step_device.cuh"
#include "step_internal.h"

namespace w12 {

struct AttPlan {
    int np;          // tiles of a prefix unit
    int per_head;    // tiles of a head
    const int *cum;  // [R + 1] tiles of the requests before r (one row tile each)
};

struct AttSeg {
    int head, unit;        // unit: global index
    int req;               // table row
    int row0, nrows;       // query rows
    int tile, left;        // key tile, tiles of the unit from here on
    int key_begin, key_end;
};

__device__ __forceinline__ int att_len(const AttendArgs &a, int r) {
    int n = a.kv_len[r];
    const int64_t room = a.table_cols << a.page_log2;
    const int cap = room < a.max_len ? int(room) : a.max_len;
    return n < 0 ? 0 : n > cap ? cap : n;
}

// Tiles of request r beyond the prefix, and of the prefix for a batch whose
// longest request has `longest` keys.
__device__ __forceinline__ int att_req_tiles(const AttendArgs &a, int len) {
    return len > a.prefix ? (len + kAttTile - 1) / kAttTile - a.prefix / kAttTile : 0;
}
__device__ __forceinline__ int att_prefix_end(const AttendArgs &a, int longest) { return min(a.prefix, longest); }

// CTA c's tiles begin at att_begin(total, grid, c); the CTA that has tile t.
__device__ __forceinline__ int att_begin(int total, int grid, int c) {
    const int per = total / grid, rem = total % grid;
    return c * per + min(c, rem);
}
__device__ __forceinline__ int att_owner(int total, int grid, int t) {
    const int per = total / grid, rem = total % grid;
    return t < rem * (per + 1) ? t / (per + 1) : rem + (t - rem * (per + 1)) / per;
}

// The request of tile w of the request part of a head (w counts tiles of one
// row tile each): the last r with cum[r] <= w.
__device__ __forceinline__ int att_find(const int *cum, int R, int w) {
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= w) lo = mid; else hi = mid;
    }
    return lo;
}

// The unit and key tile of tile t of the line.  lens: clamped lengths (shared memory).
__device__ __forceinline__ AttSeg att_locate(const AttendArgs &a, const AttPlan &p, const int *lens, int longest,
                                             int t) {
    AttSeg s;
    s.head = t / p.per_head;
    int w = t - s.head * p.per_head;
    const int per_head_units = a.pu + a.R * a.su;
    if (w < a.pu * p.np) {
        const int u = w / p.np;
        s.unit = s.head * per_head_units + u;
        s.req = 0;
        s.row0 = u * a.rt;
        s.nrows = min(a.rt, a.rows - s.row0);
        s.tile = w - u * p.np;
        s.left = p.np - s.tile;
        s.key_begin = 0;
        s.key_end = att_prefix_end(a, longest);
    } else {
        w -= a.pu * p.np;
        const int r = att_find(p.cum, a.R, w / a.su);
        const int n = p.cum[r + 1] - p.cum[r];
        w -= p.cum[r] * a.su;
        const int u = w / n, tg = a.T * a.G;
        s.unit = s.head * per_head_units + a.pu + r * a.su + u;
        s.req = r;
        s.row0 = r * tg + u * a.rt;
        s.nrows = min(a.rt, tg - u * a.rt);
        s.tile = a.prefix / kAttTile + (w - u * n);
        s.left = n - (w - u * n);
        s.key_begin = a.prefix;
        s.key_end = lens[r];
    }
    return s;
}

}  // namespace w12
