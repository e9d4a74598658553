// abi_draft.cu -- the extern "C" entry points of the calls around a draft
// model (include/w12.h: add and norm, 4-bit products, sampled verification):
// argument checks and dispatch.  Host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "draft_internal.h"

namespace w12 {

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kLim31 = int64_t(1) << 31;

size_t size_of(int dtype) { return dtype == W12_F32 ? 4 : dtype == W12_BF16 ? 2 : 1; }

bool float_type(int dtype) { return dtype == W12_F32 || dtype == W12_BF16; }

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

// SM count and CTAs per SM of a product variant on the current device, asked
// once per device and variant.
std::atomic<uint64_t> g_fp4[kMaxDevices][kFp4Variants];

int fp4_device(int variant, int *sms, int *blocks) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return W12_ERR_CUDA;
    uint64_t v = g_fp4[dev][variant].load(std::memory_order_acquire);
    if (v == 0) {
        int s = 0, b = 0;
        if (device_sm_count(&s) != W12_OK || fp4_occupancy(variant, &b) != W12_OK || b < 1) return W12_ERR_CUDA;
        v = uint64_t(s) << 32 | uint64_t(b);
        g_fp4[dev][variant].store(v, std::memory_order_release);
    }
    *sms = int(v >> 32), *blocks = int(v & 0xFFFFFFFFu);
    return W12_OK;
}

int check_fp4_shape(int64_t K, int64_t N) {
    if (K < kGroup || N < 1 || K % kGroup != 0 || K >= kLim31 || N >= kLim31) return W12_ERR_SHAPE;
    // units (and the threads that write them, one a column) in 32 bits
    return (N + kFp4Tile - 1) / kFp4Tile < (int64_t(1) << 31) / (K / kGroup) / 2 ? W12_OK : W12_ERR_SHAPE;
}

uint64_t fp4_units(int64_t K, int64_t N) { return uint64_t((N + kFp4Tile - 1) / kFp4Tile) * uint64_t(K / kGroup); }

bool usable_scale(float s) { return s >= 0x1p-100f && s <= 0x1p100f; }

constexpr size_t kFp4Counters = 4096;  // (the same for all sizes: one workspace serves them all)

struct Fp4Plan {
    int64_t U, ubase[kMaxBatch];
    size_t partial, x[kMaxBatch], total;
    int grid, grain;
};

int plan_fp4(const w12_fp4 *w, int count, int64_t M, Fp4Plan *p) {
    if (!w) return W12_ERR_ARG;
    if (count < 1 || count > kMaxBatch || M < 1 || M > W12_MAX_M) return W12_ERR_SHAPE;
    p->U = 0;
    for (int i = 0; i < count; ++i) {
        const int st = check_fp4_shape(w[i].K, w[i].N);
        if (st != W12_OK) return st;
        p->ubase[i] = p->U;
        p->U += int64_t(fp4_units(w[i].K, w[i].N));
    }
    if (p->U >= kLim31) return W12_ERR_SHAPE;
    int sms = 0, blocks = 0;
    if (fp4_device(fp4_variant(M), &sms, &blocks) != W12_OK) return W12_ERR_CUDA;
    // Equal shares of the units, or of whole tiles where their rounding costs less than
    // the fix-up of split tiles does, in units: 128 tokens 10 us of 0.9 (136 tiles of 40
    // units on 152 SMs: 35.8 units a CTA and the fix-up 57 us, 40 without 46), 32
    // tokens 5 of 0.8, one token 3 of 1.
    const int64_t ctas = int64_t(sms) * blocks, tiles = count == 1 ? (w[0].N + kFp4Tile - 1) / kFp4Tile : 0;
    const int64_t KG = w[0].K / kGroup, split = (p->U + ctas - 1) / ctas + 3 + M / 16;
    const bool whole = tiles && (tiles + ctas - 1) / ctas * KG <= split;
    p->grain = whole ? int(KG) : 1;
    p->grid = int(std::min<int64_t>(ctas, whole ? tiles : p->U));
    if (size_t(p->grid) * 4u > kFp4Counters) return W12_ERR_CUDA;
    p->partial = kWsHeader + kFp4Counters;
    size_t off = p->partial + round256(uint64_t(p->grid) * 2u * uint64_t(M) * kFp4Tile * 4u);
    for (int i = 0; i < count; ++i) {  // the tokens in bf16, where they come in e4m3
        p->x[i] = off;
        if (fp4_variant(M) >= kFp4TcVariant) off += round256(uint64_t(M) * uint64_t(w[i].K) * 2u);
    }
    p->total = off;
    return W12_OK;
}

}  // namespace

}  // namespace w12

using namespace w12;

extern "C" int w12_add_norm(const void *x, int64_t x_stride, int x_dtype, const void *delta, int64_t delta_stride,
                            int delta_dtype, const void *weight, int weight_dtype, float offset, float eps, int64_t rows,
                            int64_t dim, void *residual, int64_t residual_stride, void *out, int64_t out_stride,
                            int out_dtype, float *scale, void *stream) {
    if (!float_type(x_dtype) || (delta && !float_type(delta_dtype)) || (weight && !float_type(weight_dtype)) ||
        (out_dtype != W12_BF16 && out_dtype != W12_E4M3))
        return W12_ERR_ARG;
    if (!(eps >= 0.0f) || !(offset - offset == 0.0f) || !(eps - eps == 0.0f)) return W12_ERR_ARG;
    if (rows < 0 || rows >= kLim31 || dim < 1 || dim > W12_NORM_MAX_DIM) return W12_ERR_SHAPE;
    if (rows > 1 && (out_stride < dim || (residual && residual_stride < dim))) return W12_ERR_SHAPE;
    if (rows == 0) return W12_OK;
    if (!x || !out || (out_dtype == W12_E4M3) != (scale != nullptr)) return W12_ERR_ARG;
    if (!aligned(x, size_of(x_dtype)) || (delta && !aligned(delta, size_of(delta_dtype))) ||
        (weight && !aligned(weight, size_of(weight_dtype))) || (residual && !aligned(residual, size_of(x_dtype))) ||
        !aligned(out, size_of(out_dtype)) || !aligned(scale, 4))
        return W12_ERR_ALIGN;
    NormArgs a = {};
    a.x = x, a.delta = delta, a.weight = weight, a.residual = residual, a.out = out, a.scale = scale;
    a.x_stride = x_stride, a.delta_stride = delta_stride, a.residual_stride = residual_stride, a.out_stride = out_stride;
    a.rows = rows, a.dim = int32_t(dim), a.weight_f32 = weight && weight_dtype == W12_F32;
    a.eps = eps, a.offset = offset;
    int sms = 0;
    if (current_sms(&sms) != W12_OK) return W12_ERR_CUDA;
    a.sms = sms;
    // rows on 16-byte boundaries (e4m3: 8), whole eights of elements
    const auto rows_at = [&](const void *p, int64_t stride, size_t size, size_t to) {
        return !p || (aligned(p, to) && (rows == 1 || uint64_t(stride) * size % to == 0));
    };
    const bool vec = dim % 8 == 0 && rows_at(x, x_stride, size_of(x_dtype), 16) &&
                     rows_at(delta, delta_stride, size_of(delta_dtype), 16) && aligned(weight, 16) &&
                     rows_at(residual, residual_stride, size_of(x_dtype), 16) &&
                     rows_at(out, out_stride, size_of(out_dtype), out_dtype == W12_E4M3 ? 8 : 16);
    return launch_norm(a, x_dtype, delta ? delta_dtype : -1, out_dtype, vec, stream);
}

extern "C" size_t w12_fp4_bytes(int64_t K, int64_t N) {
    return check_fp4_shape(K, N) == W12_OK ? size_t(fp4_units(K, N)) * kFp4Unit : 0;
}

extern "C" int w12_fp4_pack(const uint8_t *codes, const uint8_t *scales, int64_t K, int64_t N, void *blob, void *stream) {
    const int st = check_fp4_shape(K, N);
    if (st != W12_OK) return st;
    if (!codes || !scales || !blob) return W12_ERR_ARG;
    if (!aligned(codes, 16) || !aligned(scales, 8) || !aligned(blob, 256)) return W12_ERR_ALIGN;
    return launch_fp4_pack(codes, scales, K, N, blob, stream);
}

extern "C" int w12_fp4_encode(const uint16_t *w, int64_t K, int64_t N, float scale, void *blob, void *stream) {
    const int st = check_fp4_shape(K, N);
    if (st != W12_OK) return st;
    if (!w || !blob || !usable_scale(scale)) return W12_ERR_ARG;
    if (!aligned(w, 16) || !aligned(blob, 256)) return W12_ERR_ALIGN;
    return launch_fp4_encode(w, K, N, scale, blob, stream);
}

extern "C" int w12_fp4_decode(const w12_fp4 *w, float *out, void *stream) {
    if (!w) return W12_ERR_ARG;
    const int st = check_fp4_shape(w->K, w->N);
    if (st != W12_OK) return st;
    if (!w->blob || !out || !usable_scale(w->scale)) return W12_ERR_ARG;
    if (!aligned(w->blob, 256) || !aligned(out, 16)) return W12_ERR_ALIGN;
    return launch_fp4_decode(w->blob, w->K, w->N, w->scale, out, stream);
}

extern "C" size_t w12_fp4_gemm_workspace_size(const w12_fp4 *w, int count, int64_t M) {
    Fp4Plan p;
    return plan_fp4(w, count, M, &p) == W12_OK ? p.total : 0;
}

extern "C" int w12_fp4_gemm_batched(const w12_fp4 *w, const void *const *x, int x_dtype, const float *const *x_scale, int64_t M,
                                    void *const *y, int y_dtype, int count, void *ws, size_t ws_bytes, int options,
                                    void *stream) {
    if ((x_dtype != W12_BF16 && x_dtype != W12_E4M3) || !float_type(y_dtype) || (options & ~W12_OPT_EARLY_WEIGHTS))
        return W12_ERR_ARG;
    const bool e4m3 = x_dtype == W12_E4M3;
    if (!w || !x || !y || e4m3 != (x_scale != nullptr)) return W12_ERR_ARG;
    if (count < 1 || count > kMaxBatch || M < 1 || M > W12_MAX_M) return W12_ERR_SHAPE;
    for (int i = 0; i < count; ++i) {
        const int st = check_fp4_shape(w[i].K, w[i].N);
        if (st != W12_OK) return st;
        if (!w[i].blob || !x[i] || !y[i] || (e4m3 && !x_scale[i]) || !usable_scale(w[i].scale)) return W12_ERR_ARG;
        if (!aligned(w[i].blob, 256) || !aligned(x[i], 16) || !aligned(y[i], size_of(y_dtype)) ||
            (e4m3 && !aligned(x_scale[i], 4)))
            return W12_ERR_ALIGN;
    }
    if (!ws) return W12_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return W12_ERR_ALIGN;
    Fp4Plan p;
    const int st = plan_fp4(w, count, M, &p);
    if (st != W12_OK) return st;
    if (ws_bytes < p.total) return W12_ERR_WORKSPACE;
    uint8_t *at = static_cast<uint8_t *>(ws);
    Fp4Batch b = {};
    for (int i = 0; i < count; ++i) {
        Fp4One &g = b.g[i];
        g.units = static_cast<const uint8_t *>(w[i].blob);
        g.x = x[i], g.x_scale = e4m3 ? x_scale[i] : nullptr, g.y = y[i];
        g.scale = w[i].scale;
        g.K = int32_t(w[i].K), g.N = int32_t(w[i].N), g.KG = int32_t(w[i].K / kGroup);
        g.NB = int32_t((w[i].N + kFp4Tile - 1) / kFp4Tile);
        g.ubase = int32_t(p.ubase[i]);
    }
    b.partial = reinterpret_cast<float *>(at + p.partial);
    b.counters = reinterpret_cast<uint32_t *>(at + kWsHeader);
    b.err = reinterpret_cast<int *>(at);
    b.count = count, b.M = int(M), b.y_dtype = y_dtype, b.U = int32_t(p.U), b.grain = p.grain;
    b.early_weights = (options & W12_OPT_EARLY_WEIGHTS) != 0;
    if (fp4_variant(M) < kFp4TcVariant) return launch_fp4(b, e4m3, p.grid, stream);
    if (e4m3)
        for (int i = 0; i < count; ++i) {
            int again = 0;  // (products that share their tokens, in rows of one length, share the copy)
            while (again < i && (x[again] != x[i] || w[again].K != w[i].K)) ++again;
            b.g[i].x = at + p.x[again];
            if (again < i) continue;
            const int done = launch_fp4_widen(x[i], at + p.x[i], M * w[i].K, stream);
            if (done != W12_OK) return done;
        }
    return launch_fp4_tc(b, p.grid, stream);
}

extern "C" int w12_fp4_gemm(const w12_fp4 *w, const void *x, int x_dtype, const float *x_scale, int64_t M, void *y, int y_dtype,
                            void *ws, size_t ws_bytes, int options, void *stream) {
    return w12_fp4_gemm_batched(w, &x, x_dtype, x_scale ? &x_scale : nullptr, M, &y, y_dtype, 1, ws, ws_bytes, options, stream);
}

namespace {

bool cut_aligned(const w12_cut *c) {
    return !c || (aligned(c->temperature, 4) && aligned(c->top_k, 4) && aligned(c->top_p, 4) && aligned(c->min_p, 4));
}

CutSide cut_side(const void *logits, int dtype, int64_t R, int64_t T, int64_t V, const w12_cut *cut, const int32_t *draft,
                 int64_t drafts, RowCut *out) {
    CutSide s = {};
    s.draft = draft, s.drafts = drafts;
    s.x = logits, s.f32 = dtype == W12_F32;
    s.vec = aligned(logits, 16) && uint64_t(V) * size_of(dtype) % 16 == 0;
    s.rows = R * T, s.T = T;
    if (cut) s.temperature = cut->temperature, s.top_k = cut->top_k, s.top_p = cut->top_p, s.min_p = cut->min_p;
    s.out = out;
    return s;
}

}  // namespace

namespace {

struct VerifyPlan {
    size_t cuts, arrived, parts, total;
    int32_t each, pieces;
};

int plan_verify(int64_t R, int64_t T, int64_t V, VerifyPlan *p) {
    if (R < 1 || T < 1 || V < 1 || V > W12_SAMPLE_MAX_V || R >= kLim31 || T >= kLim31 || R * T >= (int64_t(1) << 26))
        return W12_ERR_SHAPE;
    accept_pieces(R, V, &p->each, &p->pieces);
    p->cuts = kWsHeader;
    p->arrived = p->cuts + round256(uint64_t(R) * uint64_t(2 * T - 1) * sizeof(RowCut));
    p->parts = p->arrived + round256(uint64_t(R) * 4u);
    p->total = p->parts + round256(uint64_t(R) * uint64_t(p->pieces) * uint64_t(kAcceptRuns) * 16u);
    return W12_OK;
}

}  // namespace

extern "C" size_t w12_verify_sampled_workspace_size(int64_t R, int64_t T, int64_t V) {
    VerifyPlan p;
    return plan_verify(R, T, V, &p) == W12_OK ? p.total : 0;
}

extern "C" int w12_verify_sampled(const void *logits, int dtype, const void *draft_logits, int draft_dtype, int64_t R, int64_t T,
                                  int64_t V, const int32_t *draft, const w12_cut *target_cut, const w12_cut *draft_cut,
                                  const float *u, float *ratio, int32_t *accept_len, int32_t *next_tok, void *ws,
                                  size_t ws_bytes, void *stream) {
    if (!float_type(dtype) || (T > 1 && !float_type(draft_dtype))) return W12_ERR_ARG;
    VerifyPlan p;
    const int st = plan_verify(R, T, V, &p);
    if (st != W12_OK) return st;
    if (!logits || !u || !accept_len || !next_tok || (T > 1 && (!draft_logits || !draft))) return W12_ERR_ARG;
    if (!aligned(logits, size_of(dtype)) || (T > 1 && !aligned(draft_logits, size_of(draft_dtype))) || !aligned(u, 4) ||
        !aligned(ratio, 4) || !aligned(draft, 4) || !aligned(accept_len, 4) || !aligned(next_tok, 4) || !cut_aligned(target_cut) ||
        !cut_aligned(draft_cut))
        return W12_ERR_ALIGN;
    if (!ws || ws_bytes < p.total) return W12_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return W12_ERR_ALIGN;
    AcceptArgs a = {};
    a.logits = logits, a.draft_logits = draft_logits;
    a.f32 = dtype == W12_F32, a.draft_f32 = draft_dtype == W12_F32;
    uint8_t *w = static_cast<uint8_t *>(ws);
    RowCut *cuts = reinterpret_cast<RowCut *>(w + p.cuts);
    a.cuts = cuts, a.draft_cuts = cuts + R * T;
    a.draft = draft, a.u = u, a.ratio = ratio, a.accept_len = accept_len, a.next_tok = next_tok;
    a.R = R, a.T = T, a.V = V;
    a.arrived = reinterpret_cast<uint32_t *>(w + p.arrived);
    a.parts = reinterpret_cast<ulonglong2 *>(w + p.parts);
    a.each = p.each, a.pieces = p.pieces;
    CutArgs c = {};
    c.side[0] = cut_side(logits, dtype, R, T, V, target_cut, draft, T - 1, cuts);
    if (T > 1) c.side[1] = cut_side(draft_logits, draft_dtype, R, T - 1, V, draft_cut, draft, T - 1, cuts + R * T);
    c.V = V, c.err = reinterpret_cast<int *>(w), c.arrived = a.arrived;
    c.cuts = c.side[0].top_k || c.side[0].top_p || c.side[1].top_k || c.side[1].top_p;
    const int done = launch_cut(c, stream);
    return done == W12_OK ? launch_accept(a, stream) : done;
}
