// abi_step.cu -- the extern "C" entry points of the decode-step calls
// (include/w12.h: paged cache, attention, sampling): argument checks and
// dispatch.  Host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "step_internal.h"

namespace w12 {

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int kMaxDevices = 256;
std::atomic<int> g_sms[kMaxDevices];

// SM count of the current device, asked once per device.
int current_sms(int *sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return W12_ERR_CUDA;
    int v = g_sms[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        if (device_sm_count(&v) != W12_OK) return W12_ERR_CUDA;
        g_sms[dev].store(v, std::memory_order_relaxed);
    }
    *sms = v;
    return W12_OK;
}

int log2_of(int v) {
    int l = 0;
    while ((1 << l) < v) ++l;
    return l;
}

int check_kv(const w12_kv *kv) {
    if (!kv || (kv->dtype != W12_KV_BF16 && kv->dtype != W12_KV_E4M3)) return W12_ERR_ARG;
    if (kv->heads < 1 || kv->n_pages < 1 || (kv->head_dim != 64 && kv->head_dim != 128)) return W12_ERR_SHAPE;
    if (kv->page != 16 && kv->page != 32 && kv->page != 64 && kv->page != 128) return W12_ERR_SHAPE;
    if (kv->n_pages >= ((int64_t(1) << 31) / kv->page + kv->heads - 1) / kv->heads) return W12_ERR_SHAPE;
    const bool q8 = kv->dtype == W12_KV_E4M3;
    if (!kv->k || !kv->v || (q8 && (!kv->k_scale || !kv->v_scale))) return W12_ERR_ARG;
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || (q8 && (!aligned(kv->k_scale, 16) || !aligned(kv->v_scale, 16))))
        return W12_ERR_ALIGN;
    return W12_OK;
}

constexpr int64_t kLim31 = int64_t(1) << 31;

constexpr size_t kWsCounters = 4096;

struct AttendPlan {
    int32_t rows, sms;
    struct Line {
        int32_t pu, su, rt, halves, grid;
        size_t off_ml, off_o;
    } line[kLines];
    size_t off_arrived, off_plan, total;
    bool join;
};

// Rows per key head and request from which the tensor-memory kernel takes
// the requests: its tile has 128 rows whatever their number, the register
// kernel's work grows with them.  8 requests of 700 .. 9000 keys, 8 key heads
// (us, bf16 / e4m3), register kernel against the other: 12 rows 41 / 36
// against 47 / 62, 18 rows 56 / 67 against 46 / 60, 30 rows 60 / 73 against
// 45 / 56; of 200 .. 900 keys: 12 rows 17 / 17 against 20 / 27, 18 rows 22 /
// 33 against 20 / 26.  (The prefix of two or more requests always goes there:
// it is what reads it once.)
constexpr int64_t kTcRows = 17;

// Work split and workspace layout of an attention call.
int plan_attend(const w12_kv *kv, int64_t R, int64_t T, int q_heads, int64_t max_len, int64_t prefix, AttendPlan *p) {
    const int st = check_kv(kv);
    if (st != W12_OK) return st;
    if (R < 1 || R > W12_ATTEND_MAX_R || T < 1 || T >= kLim31 || q_heads < 1 || q_heads > (1 << 20) ||
        q_heads % kv->heads != 0)
        return W12_ERR_SHAPE;
    // (the end of a tile is a 32-bit number, too)
    if (max_len < 0 || max_len > kLim31 - 256 || prefix < 0 || prefix >= kLim31) return W12_ERR_SHAPE;
    const int64_t tg = T * (q_heads / kv->heads), rows = R * tg;
    if (rows >= kLim31 / 2) return W12_ERR_SHAPE;
    p->rows = int32_t(rows);
    const auto blocks = [](int64_t n, int64_t rt) { return int32_t((n + rt - 1) / rt); };
    auto *l = p->line;
    for (int i = 0; i < kLines; ++i) l[i] = {};
    const int64_t shared = std::min(prefix, max_len) / kAttTcTile;  // at most these many whole tiles of the prefix
    if (R > 1 && shared > 0) {
        l[kLinePrefix].rt = rows <= 128 ? 128 : 256;
        l[kLinePrefix].pu = blocks(rows, l[kLinePrefix].rt);
    }
    if (tg >= kTcRows) {
        l[kLineRequests].rt = tg <= 128 ? 128 : 256;
        l[kLineRequests].su = blocks(tg, l[kLineRequests].rt);
    } else {
        l[kLineRest].rt = tg <= 8 ? 8 : 16;
        l[kLineRest].su = 1;
    }
    const int64_t own = max_len / kAttTile + 1;  // at most these many tiles of a request
    for (int i = 0; i < kLines; ++i) {           // 32-bit tile numbers
        if (own > kLim31 / (R * std::max(l[i].su, 1)) || shared > kLim31 / std::max(l[i].pu, 1) ||
            own * R * l[i].su + shared * l[i].pu >= kLim31 / kv->heads)
            return W12_ERR_SHAPE;
    }
    int sms = 0;
    if (current_sms(&sms) != W12_OK) return W12_ERR_CUDA;
    size_t off = kWsHeader;
    p->off_arrived = off;
    off += kWsCounters;  // (the same for all sizes: one workspace serves them all)
    if (uint64_t(2 * sms) * 4u > kWsCounters) return W12_ERR_CUDA;
    p->sms = sms;
    p->off_plan = off;
    off += round256(uint64_t(R + 4) * 4u);
    p->join = l[kLinePrefix].pu + l[kLineRequests].su > 0;
    for (int i = 0; i < kLines; ++i) {
        auto &n = l[i];
        if (n.pu + n.su == 0) continue;
        n.halves = i != kLineRest && n.rt == 128 ? 2 : 1;
        const int64_t tiles = own * R * n.su + shared * n.pu;
        // (the register kernel has two workers per CTA)
        const int64_t per = i == kLineRest ? 2 : 1;
        n.grid = int(per * std::max<int64_t>(1, std::min<int64_t>(sms, (tiles * kv->heads + per - 1) / per)));
        const uint64_t rowsets = uint64_t(kv->heads * (n.pu + R * n.su) + n.grid) * n.halves * n.rt;
        n.off_ml = off;
        off += round256(rowsets * 8u);
        n.off_o = off;
        off += round256(rowsets * uint64_t(kv->head_dim) * 4u);
    }
    p->total = off;
    return W12_OK;
}

}  // namespace

}  // namespace w12

using namespace w12;

extern "C" int w12_kv_append(const w12_kv *kv, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                             const void *v, int64_t v_stride, int x_dtype, int64_t R, int64_t T, int q_heads,
                             const int32_t *table, int64_t blocks, const int32_t *kv_len, const float *rope,
                             int64_t rope_positions, int rot, int layout, uint16_t *q_out, int64_t q_out_stride,
                             int *err, void *stream) {
    int st = check_kv(kv);
    if (st != W12_OK) return st;
    if (x_dtype != W12_F32 && x_dtype != W12_BF16) return W12_ERR_ARG;
    if (layout != W12_ROPE_HALF && layout != W12_ROPE_INTERLEAVED) return W12_ERR_ARG;
    if (R < 0 || T < 1 || T >= kLim31 || R >= kLim31 || q_heads < 1 || q_heads > (1 << 20) ||
        kv->heads > (1 << 20) || blocks < 0)
        return W12_ERR_SHAPE;
    if (rot < 0 || rot % 8 != 0 || rot > kv->head_dim || rope_positions < 0) return W12_ERR_SHAPE;
    if (R * T >= kLim31) return W12_ERR_SHAPE;
    if (R == 0) return W12_OK;
    if (!q || !k || !v || !table || !kv_len || !q_out || (rot > 0 && !rope)) return W12_ERR_ARG;
    const uintptr_t xa = x_dtype == W12_F32 ? 16 : 8;  // four channels at a time
    if (!aligned(q, xa) || !aligned(k, xa) || !aligned(v, xa) || !aligned(q_out, 16) || !aligned(table, 4) ||
        !aligned(kv_len, 4) || (rot > 0 && !aligned(rope, 16)) || (err && !aligned(err, 4)))
        return W12_ERR_ALIGN;
    if (((q_stride | k_stride | v_stride) & 3) || (q_out_stride & 7)) return W12_ERR_ALIGN;
    int sms = 0;
    if (current_sms(&sms) != W12_OK) return W12_ERR_CUDA;
    AppendArgs a = {};
    a.q = q, a.k = k, a.v = v;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.out_stride = q_out_stride;
    a.q_out = q_out;
    a.kc = kv->k, a.vc = kv->v, a.ks = kv->k_scale, a.vs = kv->v_scale;
    a.table = table, a.kv_len = kv_len, a.rope = rope;
    a.rope_positions = rope_positions, a.tokens = R * T, a.table_cols = blocks, a.n_pages = kv->n_pages;
    a.T = int32_t(T), a.q_heads = q_heads, a.heads = kv->heads, a.page = kv->page, a.page_log2 = log2_of(kv->page);
    a.rot = rot, a.interleaved = layout == W12_ROPE_INTERLEAVED;
    a.err = err;
    return launch_append(a, x_dtype, kv->head_dim, kv->dtype, sms, stream);
}

extern "C" int w12_kv_read(const w12_kv *kv, const int32_t *table, int64_t blocks, const int32_t *cu_len, int64_t R,
                           int64_t tokens, uint16_t *k_out, uint16_t *v_out, int *err, void *stream) {
    int st = check_kv(kv);
    if (st != W12_OK) return st;
    if (R < 0 || tokens < 0 || R >= kLim31 || tokens >= kLim31 || blocks < 0 || kv->heads > (1 << 16))
        return W12_ERR_SHAPE;
    if (tokens == 0) return W12_OK;
    if (R == 0) return W12_ERR_SHAPE;
    if (!table || !cu_len || !k_out || !v_out) return W12_ERR_ARG;
    if (!aligned(table, 4) || !aligned(cu_len, 4) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
        (err && !aligned(err, 4)))
        return W12_ERR_ALIGN;
    int sms = 0;
    if (current_sms(&sms) != W12_OK) return W12_ERR_CUDA;
    ReadArgs a = {};
    a.kc = kv->k, a.vc = kv->v, a.ks = kv->k_scale, a.vs = kv->v_scale;
    a.table = table, a.cu_len = cu_len, a.k_out = k_out, a.v_out = v_out;
    a.R = R, a.tokens = tokens, a.table_cols = blocks, a.n_pages = kv->n_pages;
    a.heads = kv->heads, a.page = kv->page, a.page_log2 = log2_of(kv->page);
    a.err = err;
    return launch_read(a, kv->head_dim, kv->dtype, sms, stream);
}

extern "C" size_t w12_attend_workspace_size(const w12_kv *kv, int64_t R, int64_t T, int q_heads, int64_t max_len,
                                            int64_t prefix_len) {
    AttendPlan p;
    return plan_attend(kv, R, T, q_heads, max_len, prefix_len, &p) == W12_OK ? p.total : 0;
}

extern "C" int w12_attend(const w12_kv *kv, const uint16_t *q, int64_t q_stride, int64_t R, int64_t T, int q_heads,
                          const int32_t *table, int64_t blocks, const int32_t *kv_len, int64_t max_len,
                          int64_t prefix_len, float scale, uint16_t *out, int64_t out_stride, float *lse, void *ws,
                          size_t ws_bytes, void *stream) {
    if (!kv || !q || !table || !kv_len || !out || !(scale == scale)) return W12_ERR_ARG;
    if (blocks < 0) return W12_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 8) || !aligned(table, 4) || !aligned(kv_len, 4) || (lse && !aligned(lse, 4)) ||
        (q_stride & 7) || (out_stride & 3))
        return W12_ERR_ALIGN;
    AttendPlan p;
    int st = plan_attend(kv, R, T, q_heads, max_len, prefix_len, &p);
    if (st != W12_OK) return st;
    if (!ws || ws_bytes < p.total) return W12_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return W12_ERR_ALIGN;
    uint8_t *w = static_cast<uint8_t *>(ws);
    AttendArgs a = {};
    st = attend_make_maps(a, kv);
    if (st != W12_OK) return st;
    a.q = q, a.out = out, a.lse = lse;
    a.ks = kv->k_scale, a.vs = kv->v_scale;
    a.table = table, a.kv_len = kv_len;
    a.q_stride = q_stride, a.out_stride = out_stride;
    a.n_pages = kv->n_pages, a.table_cols = blocks;
    a.R = int32_t(R), a.T = int32_t(T), a.G = q_heads / kv->heads, a.heads = kv->heads;
    a.page = kv->page, a.page_log2 = log2_of(kv->page);
    a.rows = p.rows;
    a.prefix = int32_t(prefix_len), a.max_len = int32_t(max_len);
    a.scale_log2 = scale * 1.4426950408889634f;
    a.err = reinterpret_cast<int *>(w);
    a.arrived = reinterpret_cast<uint32_t *>(w + p.off_arrived);
    a.plan = reinterpret_cast<int32_t *>(w + p.off_plan);
    a.join = p.join;
    // The join's warps share entries where a row has many of them (about the
    // workers per unit, and one at either end) and there are few rows: 76
    // entries of 128 rows took 10 us in 128 warps.
    int64_t entries = 0, warps = int64_t((p.rows + 31) / 32) * kv->heads * (kv->head_dim / 4);
    for (const auto &n : p.line)
        if (n.grid) entries += (n.grid / (int64_t(kv->heads) * (n.pu + R * n.su)) + 2) * n.halves;
    a.split = 1;
    while (a.split < 8 && entries > 12 * a.split && warps * a.split * 2 <= int64_t(p.sms) * 32) a.split *= 2;
    a.sms = p.sms;
    a.per_g = ~uint64_t(0) / uint64_t(a.G) + 1;
    for (int i = 0; i < kLines; ++i) {
        const auto &n = p.line[i];
        a.line[i] = {n.pu, n.su, n.rt, n.halves, n.grid, reinterpret_cast<float *>(w + n.off_o),
                     reinterpret_cast<float2 *>(w + n.off_ml)};
    }
    for (int i = 0; i < kLines; ++i) {
        a.self = i;
        if (!a.line[i].grid) continue;
        st = i == kLineRest ? launch_attend_rest(a, kv->head_dim, kv->dtype, stream)
                            : launch_attend_tc(a, kv->head_dim, kv->dtype, stream);
        if (st != W12_OK) return st;
    }
    return p.join ? launch_attend_join(a, kv->head_dim, stream) : W12_OK;
}

extern "C" size_t w12_sample_workspace_size(int64_t R, int64_t T, int64_t V) {
    if (R < 1 || T < 1 || V < 1 || V > W12_SAMPLE_MAX_V || R >= kLim31 || T >= kLim31 || R * T >= (int64_t(1) << 27))
        return 0;
    return kWsHeader + 256;
}

extern "C" int w12_sample(const void *logits, int dtype, int64_t R, int64_t T, int64_t V, const float *temperature,
                          const int32_t *top_k, const float *top_p, const float *min_p, const float *u,
                          int32_t *tokens, float *prob, const int32_t *draft, int32_t *accept_len, int32_t *next_tok,
                          void *ws, size_t ws_bytes, void *stream) {
    if (dtype != W12_F32 && dtype != W12_BF16) return W12_ERR_ARG;
    const size_t need = w12_sample_workspace_size(R, T, V);
    if (need == 0) return W12_ERR_SHAPE;
    if (!logits || !u || !tokens || (!accept_len) != (!next_tok) || (accept_len && T > 1 && !draft)) return W12_ERR_ARG;
    for (const void *p : {static_cast<const void *>(temperature), static_cast<const void *>(top_k),
                          static_cast<const void *>(top_p), static_cast<const void *>(min_p),
                          static_cast<const void *>(u), static_cast<const void *>(tokens),
                          static_cast<const void *>(prob), static_cast<const void *>(draft),
                          static_cast<const void *>(accept_len), static_cast<const void *>(next_tok)})
        if (!aligned(p, 4)) return W12_ERR_ALIGN;
    if (!aligned(logits, dtype == W12_F32 ? 4 : 2)) return W12_ERR_ALIGN;
    if (!ws || ws_bytes < need) return W12_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return W12_ERR_ALIGN;
    SampleArgs a = {};
    a.logits = logits;
    a.temperature = temperature, a.top_k = top_k, a.top_p = top_p, a.min_p = min_p, a.u = u;
    a.tokens = tokens, a.prob = prob, a.draft = draft, a.accept_len = accept_len, a.next_tok = next_tok;
    a.counter = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(ws) + kWsHeader);
    a.V = V, a.rows = R * T, a.R = R, a.T = T;
    return launch_sample(a, dtype, stream);
}
