// draft_internal.h -- declarations shared by the calls around a draft model
// (add and norm, 4-bit products, sampled verification): argument blocks of
// the kernels and their launchers.  Not installed.
#pragma once

#include <cstddef>
#include <cstdint>

#include <vector_types.h>

#include "step_internal.h"

namespace w12 {

struct NormArgs {
    const void *x, *delta, *weight;
    void *residual, *out;
    float *scale;
    int64_t x_stride, delta_stride, residual_stride, out_stride;  // elements per row
    int64_t rows;
    int32_t dim;
    int32_t weight_f32;
    int32_t sms;
    float eps, offset;
};
// delta_dtype -1: no delta.  vec: every row of every tensor starts on a
// 16-byte boundary and dim is a multiple of 8.
int launch_norm(const NormArgs &a, int x_dtype, int delta_dtype, int out_dtype, bool vec, void *stream);

// 4-bit weights.  Unit blocks as of the W12 format: unit t * KG + kg holds
// the codes and scales of 256 columns x 128 k (include/w12.h).
constexpr int kFp4Unit = W12_FP4_UNIT_BYTES;
constexpr int kFp4Tile = 256;
constexpr int kFp4Scales = kFp4Tile * 64;  // the scales' place in a unit block

struct Fp4One {
    CUtensorMap tx;        // of x in bf16, for the tcgen05 kernel: boxes of 64 k x MP tokens
    const uint8_t *units;
    const void *x;         // [M][K] bf16, or e4m3 with
    const float *x_scale;  // [M]
    void *y;               // [M][N]
    float scale;
    int32_t K, N, KG, NB;
    int32_t ubase;         // first unit of this product
};

struct Fp4Batch {
    Fp4One g[kMaxBatch];
    float *partial;      // [grid][2][M][256] partial sums of split tiles
    uint32_t *counters;  // [grid] arrivals of a split tile, by the CTA that has its first unit (zero between calls)
    int *err;
    int count, M, y_dtype;
    int32_t U;
    int32_t grain;      // units that stay together in a CTA: 1, or a tile's (nothing is split)
    int early_weights;  // the first weight copies do not wait for the kernel before
};

int launch_fp4_pack(const uint8_t *codes, const uint8_t *scales, int64_t K, int64_t N, void *blob, void *stream);
int launch_fp4_encode(const uint16_t *w, int64_t K, int64_t N, float scale, void *blob, void *stream);
int launch_fp4_decode(const void *blob, int64_t K, int64_t N, float scale, float *out, void *stream);
// The product kernels' variant for M tokens (from kFp4TcVariant on: tcgen05), and
// its CTAs per SM (the call also raises the variant's shared-memory limit on the
// current device).
constexpr int kFp4Variants = 5, kFp4TcVariant = 2;
inline int fp4_variant(int64_t M) { return M <= 8 ? 0 : M <= 16 ? 1 : M <= 32 ? 2 : M <= 64 ? 3 : 4; }
int fp4_occupancy(int variant, int *blocks);
int fp4_tc_occupancy(int variant, int *blocks);
int launch_fp4(const Fp4Batch &b, bool e4m3, int grid, void *stream);
// x of b.g[i] is bf16 here; its tensor maps are made by the call.
int launch_fp4_tc(Fp4Batch &b, int grid, void *stream);
// n e4m3 codes as bf16 (n a multiple of 16).
int launch_fp4_widen(const void *codes, void *out, int64_t n, void *stream);

// What the cuts leave of a row: the tokens with a logit above `least`, or equal
// with an index of `last` at most, whose weight (with mx and inv_t; cut_device.cuh)
// is not below `floor`.  A row whose largest logit is infinite has least = infinity
// and mx the largest float, one without any token last = -1 besides.
struct RowCut {
    float mx, inv_t, least, floor;
    int32_t last;
    int32_t one;   // >= 0: that token alone stays (it is `last`)
    float inv;     // 1 / the sum of the weights that stay; 0: none does
    float share;   // of the row's drafted token (0: there is none)
};

// The cuts of the rows of two tensors of logits (the target's, the drafter's).
struct CutSide {
    const void *x;
    int32_t f32;
    int32_t vec;         // rows on 16-byte boundaries, whole 16-byte pieces
    int64_t rows, T;     // T rows per request
    const float *temperature, *top_p, *min_p;
    const int32_t *top_k;
    const int32_t *draft;  // [requests][drafts]: of row r that of r % T, where it is below drafts
    int64_t drafts;
    RowCut *out;
};

struct CutArgs {
    CutSide side[2];
    int64_t V;
    int32_t chunk;       // logits per CTA of a row's cluster
    int32_t ahead;       // rows that the GPU holds at a time
    int32_t cuts;        // a top_k or top_p is given
    int *err;
    uint32_t *arrived;   // [requests] set to zero, for launch_accept
};
int launch_cut(CutArgs &a, void *stream);

struct AcceptArgs {
    const void *logits, *draft_logits;  // [R T][V], [R (T - 1)][V]
    int32_t f32, draft_f32;
    const RowCut *cuts, *draft_cuts;    // of their rows
    const int32_t *draft;
    const float *u;
    float *ratio;
    int32_t *accept_len, *next_tok;
    int64_t R, T, V;
    uint32_t *arrived;      // [R], zeros
    ulonglong2 *parts;      // [R][pieces * kAcceptRuns]
    int32_t each, pieces;   // tokens a CTA (a multiple of 1024), CTAs a row
};
constexpr int kAcceptRuns = 8;  // of a CTA's piece
void accept_pieces(int64_t R, int64_t V, int32_t *each, int32_t *pieces);
int launch_accept(const AcceptArgs &a, void *stream);

}  // namespace w12
