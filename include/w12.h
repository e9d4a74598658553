/*
 * w12.h -- C interface of libw12.so: the W12 lossless 12-bit BF16 weight
 * format, the fused W12 decode-GEMM for skinny M, and greedy draft-block
 * verification, for NVIDIA GB300 (sm_103a).
 *
 * Sources.  The SpecPilot summary pages (airadar.tv, English edition,
 * "Reasons" bullet 2, and its French, Japanese and Korean editions) describe
 * W12 as BF16 split into three 4-bit planes and rebuilt bit for bit inside the
 * GEMM's registers; the hotrepo.ai page on StargazerX0/SpecPilot ("项目介绍",
 * paragraph 2) adds that the decode is bit-exact and serves batch 1-32.  The
 * same English page ("Risks", bullet 3) defines the greedy acceptance rule:
 * every committed token is the target model's own greedy choice.  No layout,
 * interface or kernel is printed there; the layout and calls below are this
 * library's own.
 *
 * Conventions for every call:
 *  - Status: every function returns an int status (W12_OK = 0 or a W12_ERR_*
 *    code); w12_status_string() names it.  A non-zero status means nothing
 *    was launched or written.
 *  - Memory: the caller owns every buffer.  The library allocates no device
 *    memory and no host memory beyond stack and OpenMP temporaries.
 *  - Streams: `stream` is a cudaStream_t passed as void* (NULL = the legacy
 *    default stream).  Device calls are asynchronous on that stream and never
 *    synchronise, except w12_get_device_error().
 *  - The GEMM and fused-verify kernels use programmatic dependent launch:
 *    they may start while the kernel launched just before them on the same
 *    stream is finishing, but by default they read nothing in global memory
 *    (blob, x, hidden, draft, workspace) before that kernel has completed,
 *    so any producer of their inputs is safe.  The GEMM calls take one
 *    option, W12_OPT_EARLY_WEIGHTS (OR-ed into the path argument of the
 *    _ex calls): the first weight copies then start before the wait, under
 *    the previous kernel's tail; the caller promises that the blob was not
 *    written by the kernel launched just before the call on the same stream
 *    (another launch, an event or a synchronisation in between suffices;
 *    w12_encode_device ends with such a launch; copies and memsets are not
 *    kernels and need nothing).
 *  - Pointers named *_dev are device pointers, *_host host pointers.
 *  - Workspaces: a workspace of the size the matching *_workspace_size()
 *    call returns, 256-byte aligned, zero-filled by the caller before its
 *    first use.  Every kernel leaves its workspace counters at zero again, so
 *    the calls that a workspace belongs to reuse it without clearing:
 *    w12_gemm, w12_gemm_ex, w12_gemm_batched and w12_gemm_batched_ex with the
 *    same matrices (any M and path); w12_verify_greedy_lmhead with the same
 *    matrix and R T; w12_fp4_gemm and w12_fp4_gemm_batched; each other call by itself,
 *    in any size that needs no more than it has.  Counters lie at different
 *    places for different calls, and results on the way to the next kernel
 *    stay where they are: a workspace that passes from one of these to another
 *    has to be zero-filled in between.  Word 0 of a workspace is a
 *    sticky device error code (see w12_get_device_error).  Calls that share
 *    one workspace must be ordered (same stream, or events).
 */
#ifndef W12_H
#define W12_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define W12_FORMAT_VERSION 2

/* Status codes. */
#define W12_OK 0
#define W12_ERR_ARG 1               /* NULL pointer, bad enum, inconsistent desc   */
#define W12_ERR_SHAPE 2             /* K % 128 != 0, negative sizes, M or T range  */
#define W12_ERR_ALIGN 3             /* a pointer misses its required alignment     */
#define W12_ERR_WORKSPACE 4         /* workspace NULL or smaller than required     */
#define W12_ERR_BLOB 5              /* blob contents inconsistent with the desc    */
#define W12_ERR_TOO_MANY_ESCAPES 6  /* 2^24 or more escapes in one matrix          */
#define W12_ERR_CUDA 7              /* a CUDA runtime call or launch failed        */
#define W12_ERR_TIMEOUT 8           /* a bounded device wait gave up               */
#define W12_ERR_DEVICE 9            /* a kernel recorded an error (bad blob index) */

/* Orientation of a dense weight matrix in memory. */
#define W12_LAYOUT_KN 0 /* w[k*N + n]: row-major [K][N]                         */
#define W12_LAYOUT_NK 1 /* w[n*K + k]: row-major [N][K] (a linear layer's weight) */

/* Element types of y and of logits (and, where a call says so, of x). */
#define W12_F32 0
#define W12_BF16 1
#define W12_E4M3 2 /* 8-bit codes with one fp32 scale per row: value = code * scale */

/* GEMM paths (w12_gemm_ex, w12_gemm_batched_ex).  All three stream the
 * weights' unit blocks with bulk copies (TMA) through a shared-memory ring,
 * stream-K over the whole GPU; they differ in the contraction.
 * W12_PATH_AUTO takes the GEMV at M = 1 and tcgen05 above (the fastest on
 * GB300 from 2 tokens on). */
#define W12_PATH_AUTO 0
#define W12_PATH_GEMV 1 /* CUDA-core bf16 FMA GEMV with warp-shuffle reduction, M <= 4   */
#define W12_PATH_MMA 2  /* mma.sync tiles, M <= 128                                     */
#define W12_PATH_TC 3   /* tcgen05: weights rebuilt into tensor memory, fp32 accumulator
                           in tensor memory, M <= 128                                    */

#define W12_MAX_M 128

/* Option bit of the path argument of w12_gemm_ex / w12_gemm_batched_ex:
 * start streaming the weights before the previous kernel of the stream has
 * completed (see the conventions above).  Default off. */
#define W12_OPT_EARLY_WEIGHTS 0x100

/*
 * Descriptor of one encoded K x N matrix (format v2).
 *
 * Logical format.  A group is 128 consecutive k of one output column n
 * (pos = k % 128).  A bf16 weight has sign s (bit 15), exponent e (bits
 * 14..7) and mantissa m (bits 6..0).  Each group has a base b in [0, 240]:
 * the b whose window [b, b+14] holds the most of the group's exponents, the
 * largest such b on a tie.  A weight's exponent code is c = e - b inside the
 * window and 15 ("escape") outside it; an escaped weight gets a 16-bit entry
 * pos | e << 7 in the escape list.  Weights k and k^1 (an even k and the
 * next) form a pair; each stores its pair partner's sign.
 *
 * Physical format: plane-major, 16-byte-aligned tiles.
 *  - Columns are cut into tiles of 128 (T = ceil(N / 128) tiles; columns
 *    past N are padding) and k into groups (KG = K / 128).  Unit
 *    u = t * KG + kg holds group kg of the 128 columns of tile t; the blob
 *    starts with the U = T * KG unit blocks, each W12_UNIT_BYTES long:
 *      [0, 8192)      H plane: nibble = SM'(k) >> 4
 *      [8192, 16384)  L plane: nibble = SM'(k) & 15
 *      [16384, 24576) E plane: nibble = c(k)
 *      [24576, 25092) meta: 129 little-endian uint32
 *      [25092, 25104) zero
 *    with SM'(k) = m(k) << 1 | s(k ^ 1).
 *  - In a plane block, column c of the tile owns the 64-byte row
 *    [64 c, 64 c + 64): four 16-byte chunks, chunk j holding pos
 *    32 j .. 32 j + 31 as four little-endian 32-bit words (word q: pos
 *    32 j + 8 q + 0..7).  Logical chunk j is stored at chunk position
 *    j ^ ((c >> 1) & 3).  Nibble p (bits 4p..4p+3) of a word covering pos
 *    p0..p0+7 holds the weight p0 + P[p]:
 *      H: P = {4,0,5,1,6,2,7,3}   L: P = {0,5,1,6,2,7,3,4}   E: P = {0,4,1,5,2,6,3,7}
 *  - Meta word c < 128 = b | first_escape_index(u, c) << 8; word 128 =
 *    first_escape_index(u + 1, 0) << 8 (n_esc << 8 for the last unit), so
 *    column c's escapes in unit u are entries [word c >> 8, word c+1 >> 8).
 *    Padding columns have b = 0 and no escapes; their plane bytes are 0.
 *  - The escape list (n_esc uint16 entries, ordered by unit, then column,
 *    then pos) starts at off_esc, the first 256-byte boundary after the
 *    units.  total_bytes = off_esc + 2 n_esc rounded up to 256.
 * Every unit is one contiguous, 16-byte-aligned block (the blob itself must
 * be 256-byte aligned on the device), so a kernel streams a unit with one
 * bulk copy.
 */
#define W12_UNIT_BYTES 25104
typedef struct w12_desc {
    uint32_t version;    /* W12_FORMAT_VERSION */
    uint32_t reserved;   /* 0 */
    int64_t K, N, G;     /* G = N * K / 128 groups of real columns */
    uint64_t tiles;      /* T = ceil(N / 128) */
    uint64_t unit_bytes; /* W12_UNIT_BYTES */
    uint64_t n_units;    /* U = T * K / 128 */
    uint64_t off_units;  /* 0 */
    uint64_t off_esc;
    uint64_t n_esc;
    uint64_t total_bytes;
} w12_desc;

/* Name of a status code (static string, never NULL). */
const char *w12_status_string(int status);

/* Library format version (W12_FORMAT_VERSION). */
int w12_version(void);

/* --------------------------------------------------------------------- */
/* Host encoder                                                          */
/* --------------------------------------------------------------------- */

/*
 * Defined by: the W12 format (SpecPilot summary, airadar.tv English edition,
 * "Reasons" bullet 2: BF16 split into three 4-bit planes; hotrepo.ai
 * StargazerX0/SpecPilot page, "项目介绍" paragraph 2: lossless, decoded
 * bit-exactly).  The group size, base rule, escape list and packing are this
 * library's reading (the format description above).
 *
 * Size the blob for a bf16 matrix w (host, layout W12_LAYOUT_KN or _NK,
 * K % 128 == 0; K or N may be 0).  Fills every field of *d, counting the
 * escapes.  Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_TOO_MANY_ESCAPES.
 * Multithreaded (OpenMP) over groups.
 */
int w12_encode_plan(const uint16_t *w_host, int64_t K, int64_t N, int layout, w12_desc *d);

/*
 * Defined by: as w12_encode_plan ("Reasons" bullet 2; "项目介绍" paragraph 2).
 *
 * Encode w into blob_host (d->total_bytes bytes, any alignment; padding is
 * written as zeros).  *d must come from w12_encode_plan on the same w.
 * Errors: W12_ERR_ARG (d does not match w), W12_ERR_SHAPE.
 */
int w12_encode(const uint16_t *w_host, int64_t K, int64_t N, int layout, const w12_desc *d,
               void *blob_host);

/*
 * Defined by: the format description above (this library's reading of
 * "Reasons" bullet 2).
 *
 * Check a host blob against its descriptor: the offsets and sizes, base
 * range, meta monotonicity and sentinel, escape positions and order, that
 * every code-15 nibble has exactly one escape entry and that every escape is
 * canonical (its exponent lies outside the group window).  Returns W12_OK,
 * W12_ERR_ARG or W12_ERR_BLOB.  The device calls do not run this check:
 * they only bound every index they read, recording W12_ERR_DEVICE.
 */
int w12_validate(const w12_desc *d, const void *blob_host);

/* --------------------------------------------------------------------- */
/* Device encoder (the same bytes as the host encoder)                  */
/* --------------------------------------------------------------------- */

/* Bytes of workspace w12_encode_plan_device / w12_encode_device need for a
 * K x N matrix (>= 256; 0 for a negative size). */
size_t w12_encode_device_workspace_size(int64_t K, int64_t N);

/*
 * Defined by: as w12_encode_plan ("Reasons" bullet 2; "项目介绍" paragraph 2).
 *
 * w12_encode_plan on the GPU, for weights already in device memory (a model
 * loaded straight to HBM: no pass over the weights on the host).  w_dev: the
 * bf16 matrix in layout W12_LAYOUT_KN or _NK, 16-byte aligned.  Computes
 * every group's base and escape count into the workspace, fills *d (the
 * descriptor w12_encode_plan gives for the same matrix) and waits for
 * `stream` (the escape count is read back to size the blob).  Keep the
 * workspace for w12_encode_device.  Up to 2^24 unit columns (ceil(N/128) *
 * K/128 * 128 <= 2^24, about 2^31 weights) per matrix.
 * Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_WORKSPACE,
 * W12_ERR_TOO_MANY_ESCAPES, W12_ERR_CUDA.
 */
int w12_encode_plan_device(const uint16_t *w_dev, int64_t K, int64_t N, int layout, w12_desc *d,
                           void *ws_dev, size_t ws_bytes, void *stream);

/*
 * Defined by: as w12_encode ("Reasons" bullet 2; "项目介绍" paragraph 2).
 *
 * w12_encode on the GPU: writes the blob of *d (from w12_encode_plan_device
 * on the same w_dev, layout and workspace) into blob_dev (d->total_bytes,
 * 256-byte aligned), byte for byte what w12_encode writes.  Asynchronous on
 * `stream`.  Errors: W12_ERR_ARG (d does not match K, N), W12_ERR_ALIGN,
 * W12_ERR_WORKSPACE, W12_ERR_CUDA.
 */
int w12_encode_device(const uint16_t *w_dev, int64_t K, int64_t N, int layout, const w12_desc *d,
                      void *blob_dev, void *ws_dev, size_t ws_bytes, void *stream);

/* --------------------------------------------------------------------- */
/* Device calls                                                          */
/* --------------------------------------------------------------------- */

/*
 * Defined by: "项目介绍" paragraph 2 (W12 is decoded bit-exactly) and
 * "Reasons" bullet 2 (the three planes are rebuilt bit by bit).
 *
 * Decode a device blob (256-byte aligned) back to bf16 bit patterns in w_dev
 * (K*N uint16, 16-byte aligned) in the given layout.  Bit-exact inverse of
 * w12_encode.  Errors: W12_ERR_ARG, W12_ERR_ALIGN, W12_ERR_CUDA.  Escape
 * indices are bounds-checked; a bad one is not followed (the weight keeps
 * the garbage exponent) and W12_ERR_DEVICE goes to *err_dev if err_dev is
 * not NULL.
 */
int w12_decode(const w12_desc *d, const void *blob_dev, uint16_t *w_dev, int layout,
               int *err_dev, void *stream);

/* Bytes of workspace w12_gemm needs for this matrix and M (>= 256). */
size_t w12_gemm_workspace_size(const w12_desc *d, int64_t M);

/*
 * Defined by: "Reasons" bullet 2 (the planes are rebuilt bit by bit inside the
 * GEMM's registers) and "项目介绍" paragraph 2 (a bit-exact decode inside the
 * GEMM, batch 1-32); the first paragraph of the summary (a decode step reads
 * every weight) makes it a weight stream.
 *
 * y[m, n] = sum_k x[m, k] * W[k, n] for m < M, n < N.
 *   x_dev: [M][K] row-major bf16, 16-byte aligned.
 *   y_dev: [M][N] row-major, y_dtype W12_F32 (4-byte aligned) or W12_BF16
 *          (2-byte aligned; rounded to nearest even from the fp32 sum).
 *   1 <= M <= W12_MAX_M.  Accumulation is fp32; the summation order is fixed
 *   for a given (desc, M) so repeated calls give identical bits.
 * Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_WORKSPACE,
 * W12_ERR_CUDA.  Device-detected blob errors: W12_ERR_DEVICE in word 0 of ws.
 */
int w12_gemm(const w12_desc *d, const void *blob_dev, const uint16_t *x_dev, int64_t M,
             void *y_dev, int y_dtype, void *ws_dev, size_t ws_bytes, void *stream);

/* w12_gemm with an explicit path (W12_PATH_*, optionally OR-ed with
 * W12_OPT_EARLY_WEIGHTS); W12_ERR_SHAPE if the path does not serve this M,
 * W12_ERR_ARG for an unknown path or option bit. */
int w12_gemm_ex(const w12_desc *d, const void *blob_dev, const uint16_t *x_dev, int64_t M,
                void *y_dev, int y_dtype, void *ws_dev, size_t ws_bytes, int path,
                void *stream);

#define W12_MAX_BATCH 8

/* Bytes of workspace w12_gemm_batched (and w12_gemm_batched_ex, on any path
 * that serves this M) needs for these matrices and M (0 on invalid
 * arguments). */
size_t w12_gemm_batched_workspace_size(const w12_desc *descs, int count, int64_t M);

/*
 * Defined by: as w12_gemm ("Reasons" bullet 2; "项目介绍" paragraph 2).
 *
 * count independent products y_i = x_i . W_i (1 <= count <= W12_MAX_BATCH,
 * every K_i, N_i > 0) with one M, e.g. the linears of a decoder layer, in ONE
 * kernel launch: the work units of all products (stream-K units of columns x
 * 1024 k) are split evenly over the GPU, so small products (a layer's k and
 * v) neither run alone on a part of the SMs nor pay their own launch and
 * tail.  descs, blobs_dev, x_dev, y_dev are host arrays of count entries
 * (device pointers in the last three), with the layouts and alignments of
 * w12_gemm.  The bits of the results depend only on the descriptors, M, the
 * path and the GPU's SM count (the units' split over the CTAs fixes where
 * fp32 partial sums are cut), so repeated calls give identical results.
 * Errors: as w12_gemm; W12_ERR_SHAPE for an empty product.
 */
int w12_gemm_batched(const w12_desc *descs, const void *const *blobs_dev,
                     const uint16_t *const *x_dev, int64_t M, void *const *y_dev, int y_dtype,
                     int count, void *ws_dev, size_t ws_bytes, void *stream);

/* w12_gemm_batched with an explicit path (W12_PATH_*, optionally OR-ed with
 * W12_OPT_EARLY_WEIGHTS); W12_ERR_SHAPE if the path does not serve this M,
 * W12_ERR_ARG for an unknown path or option bit. */
int w12_gemm_batched_ex(const w12_desc *descs, const void *const *blobs_dev,
                        const uint16_t *const *x_dev, int64_t M, void *const *y_dev, int y_dtype,
                        int count, void *ws_dev, size_t ws_bytes, int path, void *stream);

/*
 * Test hooks of w12_gemm_batched_debug (no counterpart on the pages: they
 * exist to exercise the kernels' bounded waits on a GPU).
 *   withhold_unit: -1, or a work unit (0 <= unit < the batch's unit count)
 *     whose weight copy the producer never issues, so that the consumers'
 *     wait on it runs out and the call records W12_ERR_TIMEOUT.
 *   wait_limit_us: the limit of one bounded wait in microseconds (0: the
 *     default of 2 s; at most 10 s).
 */
typedef struct w12_debug_opts {
    int32_t withhold_unit;
    uint32_t wait_limit_us;
} w12_debug_opts;

/*
 * w12_gemm_batched_ex with test hooks.  With withhold_unit = -1 and
 * wait_limit_us = 0 it is w12_gemm_batched_ex.  After a withheld unit the
 * outputs are undefined and word 0 of the workspace reads W12_ERR_TIMEOUT;
 * every kernel still runs to its end (no wait is unbounded), the
 * workspace's counters are left at zero, and the next call on the same
 * workspace is correct.  Errors: as w12_gemm_batched_ex; W12_ERR_ARG for a
 * NULL dbg or a hook out of range.
 */
int w12_gemm_batched_debug(const w12_desc *descs, const void *const *blobs_dev,
                           const uint16_t *const *x_dev, int64_t M, void *const *y_dev, int y_dtype,
                           int count, void *ws_dev, size_t ws_bytes, int path,
                           const w12_debug_opts *dbg, void *stream);

/* Bytes of workspace w12_verify_greedy needs (>= 256). */
size_t w12_verify_workspace_size(int64_t R, int64_t T, int64_t V);

/*
 * Defined by: "Risks" bullet 3 of the SpecPilot summary (lossless means every
 * committed token is the target model's own greedy choice) and the
 * hotrepo.ai page's "结果与验证" (each committed token is checked against the
 * target's choice at its position).  Tie, NaN and -0 handling and the draft
 * alignment are this library's reading (the pages are silent on them).
 *
 * Greedy verification of R draft blocks of T positions on logits.
 *   logits_dev: [R*T][V] row-major, dtype W12_F32 or W12_BF16, 16-byte aligned.
 *   draft_dev:  [R][T-1] int32 (may be NULL when T == 1).
 *   For each row i of block r, g[r,i] is the lowest index of the row maximum
 *   (NaN above every number, the first NaN wins, -0 == +0).  Row i is the
 *   target's prediction after block input [last token, d0 .. d(i-1)], so it
 *   is compared with draft token i:
 *     accept_len_dev[r] = first i < T-1 with draft[r,i] != g[r,i], else T-1;
 *     next_tok_dev[r]   = g[r, accept_len[r]].
 *   R >= 1, T >= 1, 1 <= V < 2^31.
 * Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_WORKSPACE,
 * W12_ERR_CUDA.
 */
int w12_verify_greedy(const void *logits_dev, int dtype, int64_t R, int64_t T, int64_t V,
                      const int32_t *draft_dev, int32_t *accept_len_dev, int32_t *next_tok_dev,
                      void *ws_dev, size_t ws_bytes, void *stream);

/* Bytes of workspace w12_verify_greedy_lmhead needs (>= 256). */
size_t w12_verify_lmhead_workspace_size(const w12_desc *d_lm, int64_t R, int64_t T);

/*
 * Defined by: as w12_gemm (the lm_head product) and w12_verify_greedy (the
 * acceptance rule): "Reasons" bullet 2, "Risks" bullet 3, "结果与验证".
 *
 * Fused lm_head + greedy verification: logits = hidden @ W_lm (the W12
 * decode-GEMM, fp32 accumulation), then the rule of w12_verify_greedy on
 * those fp32 logits, without writing them unless logits_out_dev is given.
 *   hidden_dev: [R*T][K] bf16, 16-byte aligned; R*T <= W12_MAX_M.
 *   logits_out_dev: NULL, or [R*T][N] fp32 receiving the exact logits the
 *   argmax was taken on.
 * Errors: as w12_gemm and w12_verify_greedy.
 */
int w12_verify_greedy_lmhead(const uint16_t *hidden_dev, const w12_desc *d_lm,
                             const void *blob_lm_dev, int64_t R, int64_t T,
                             const int32_t *draft_dev, int32_t *accept_len_dev,
                             int32_t *next_tok_dev, float *logits_out_dev, void *ws_dev,
                             size_t ws_bytes, void *stream);

/*
 * Scratch memory that w12_verify_greedy_noalloc() keeps, once, on every GPU
 * that loads this library (held until the process exits).
 */
#define W12_NOALLOC_SCRATCH_BYTES (256u * 1024u)

/*
 * w12_verify_greedy() for callers that cannot allocate device memory: a
 * serving loop whose device memory is planned once and may not grow, a host
 * framework that owns every device allocation and passes only inputs and
 * outputs, or a latency-critical path that cannot afford cudaMalloc's
 * implicit device synchronisation.  The paper has no counterpart: this entry
 * point exists only for such callers.
 *
 * Same arguments and results as w12_verify_greedy() without the workspace:
 * the scratch (an arrival counter, the per-slice argmax keys and the
 * per-row tokens) is a fixed W12_NOALLOC_SCRATCH_BYTES array inside the
 * library.  The call allocates nothing, host or device.
 *  - Size limit: a call needs 512 + 8 * R*T * splits + 4 * R*T bytes (each
 *    term rounded up to 256), with splits = max(1, ceil(4 * SMs / (R*T)))
 *    capped at ceil(V / 1024); beyond W12_NOALLOC_SCRATCH_BYTES (about 20000
 *    rows of R*T) it returns W12_ERR_WORKSPACE and launches nothing.
 *  - The first call on each device looks up the array's device address
 *    (cudaGetSymbolAddress, with that device current) and caches it; make
 *    that first call before any stream capture begins.
 *  - Every call on a device shares the one array, which keeps the previous
 *    call's contents; each call clears what has to start at zero.  Calls
 *    that may overlap on the GPU (different streams without ordering, or
 *    several host threads) race on the array and give wrong results:
 *    order them.
 * Errors: as w12_verify_greedy, plus W12_ERR_WORKSPACE for the size limit.
 */
int w12_verify_greedy_noalloc(const void *logits_dev, int dtype, int64_t R, int64_t T, int64_t V,
                              const int32_t *draft_dev, int32_t *accept_len_dev,
                              int32_t *next_tok_dev, void *stream);

/* --------------------------------------------------------------------- */
/* Decode step: paged key/value cache                                    */
/* --------------------------------------------------------------------- */

/*
 * The calls from here on are the parts of a decode step between
 * the projections (w12_gemm_batched) and the committed token: rotary
 * positions and the cache write, attention over the cache, sampling.  The
 * SpecPilot pages describe no layout or rule for them; they are this
 * library's own.  They use programmatic dependent launch as the GEMM calls
 * do: nothing in global memory is read or written before the kernel launched
 * just before on the same stream has completed.
 */

/* Element types of a cache. */
#define W12_KV_BF16 0
#define W12_KV_E4M3 1 /* 8-bit codes, one fp32 scale per token and head: value = code * scale */

/*
 * A paged cache: pages of `page` tokens (16, 32, 64 or 128).
 *   k, v: [n_pages][heads][page][head_dim] bf16 or e4m3, 16-byte aligned;
 *   k_scale, v_scale: [n_pages][heads][page] fp32, 16-byte aligned
 *     (W12_KV_E4M3), else NULL.
 * head_dim is 64 or 128; n_pages * heads * page < 2^31.  Memory is the
 * caller's; rows that were never written are never looked at.
 */
typedef struct w12_kv {
    void *k, *v;
    float *k_scale, *v_scale;
    int64_t n_pages;
    int32_t heads, head_dim, page, dtype;
} w12_kv;

/*
 * Requests.  A call serves R requests of T new tokens each (T = 1: plain
 * decoding; a draft block; a piece of a prompt), tokens ordered [R][T].
 *   kv_len_dev: [R] int32, each request's length WITH its T new tokens:
 *     token i of request r has position kv_len[r] - T + i.  A negative
 *     position is a padding token (a request with fewer than T tokens).
 *   block_table_dev: [R][blocks] int32: position p of request r lives in row
 *     p % page of page block_table[r][p / page].
 * Lengths and tables stay on the device; a bad entry (a page outside
 * [0, n_pages), a position past the table) is not followed and records
 * W12_ERR_DEVICE.
 */

/* Channel pairs of a rotated head with `rot` rotated channels. */
#define W12_ROPE_HALF 0        /* pair j: channels j and j + rot / 2 */
#define W12_ROPE_INTERLEAVED 1 /* pair j: channels 2 j and 2 j + 1   */

/* Scaling of the rotary frequencies f_j = base^(-2 j / rot) for contexts
 * beyond the `original` trained length. */
#define W12_ROPE_SCALE_NONE 0
#define W12_ROPE_SCALE_LINEAR 1 /* f_j / factor                                                  */
#define W12_ROPE_SCALE_BASE 2   /* base * factor^(rot / (rot - 2)) in place of base              */
#define W12_ROPE_SCALE_BANDS 3  /* f_j (g + (1 - g) / factor), g = (turns_j - low) / (high - low)
                                   in [0, 1], turns_j = original f_j / (2 pi)                    */
#define W12_ROPE_SCALE_YARN 4   /* as BANDS with g linear in j between the (rounded outwards)
                                   channels that make `high` and `low` turns, and cos and sin
                                   times `attention` (0: 0.1 ln(factor) + 1)                     */
typedef struct w12_rope_scaling {
    int32_t mode, reserved;
    double factor;    /* > 0 */
    double original;  /* > 0; BANDS, YARN */
    double low, high; /* 0 < low < high; BANDS, YARN */
    double attention; /* >= 0; YARN */
} w12_rope_scaling;

/*
 * Rotary table on the host: table[p][0 .. rot/2) = cos(p f_j),
 * table[p][rot/2 .. rot) = sin(p f_j) for p < positions, computed in double
 * precision and rounded once.  rot: a multiple of 8; base > 1; scaling may
 * be NULL (none).  Errors: W12_ERR_ARG, W12_ERR_SHAPE.  Multithreaded.
 */
int w12_rope_table(int64_t positions, int rot, double base, const w12_rope_scaling *scaling, float *table_host);

/*
 * Rotate the queries and keys of R * T new tokens and write keys and values
 * into the cache (rounded to bf16, or quantised), in one launch.
 *   q_dev, k_dev, v_dev: x_dtype W12_F32 or W12_BF16; token n's heads start at
 *     q_dev + n * q_stride (elements; heads and channels contiguous), so the
 *     three may be parts of one projection output.  16-byte (F32) or 8-byte
 *     (BF16) aligned, strides multiples of 4.
 *   rope_dev: fp32 [rope_positions][rot] (w12_rope_table), 16-byte aligned;
 *     NULL with rot = 0: no rotation.  rot is a multiple of 8, at most
 *     head_dim; the channels from rot on are left as they are.
 *   q_out_dev: bf16, token stride q_out_stride (a multiple of 8), 16-byte
 *     aligned, not overlapping the inputs.  Padding tokens write nothing, here
 *     and in the cache.
 * W12_KV_E4M3: a row's scale is amax / 448 and its codes are
 * round(x * (448 / amax)) (nearest even); a row whose amax is at most 1e-30
 * is stored as zeros; one that holds a NaN or an infinity reads back as NaN.
 * Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_CUDA.  Device
 * errors (also a position past rope_positions) go to *err_dev if it is not
 * NULL; such a token writes nothing.
 */
int w12_kv_append(const w12_kv *kv, const void *q_dev, int64_t q_stride, const void *k_dev, int64_t k_stride,
                  const void *v_dev, int64_t v_stride, int x_dtype, int64_t R, int64_t T, int q_heads,
                  const int32_t *block_table_dev, int64_t blocks, const int32_t *kv_len_dev, const float *rope_dev,
                  int64_t rope_positions, int rot, int layout, uint16_t *q_out_dev, int64_t q_out_stride,
                  int *err_dev, void *stream);

/*
 * Read the cache back: rows 0 .. cu_len[r+1] - cu_len[r] - 1 of every
 * request, packed, as bf16 (codes times scale, rounded once).
 *   cu_len_dev: [R + 1] int32, cu_len[0] = 0, not decreasing, cu_len[R] = tokens.
 *   k_out_dev, v_out_dev: [tokens][heads][head_dim] bf16, 16-byte aligned.
 * A row whose table entry is bad reads as zeros and records W12_ERR_DEVICE
 * in *err_dev (may be NULL).
 * Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_CUDA.
 */
int w12_kv_read(const w12_kv *kv, const int32_t *block_table_dev, int64_t blocks, const int32_t *cu_len_dev,
                int64_t R, int64_t tokens, uint16_t *k_out_dev, uint16_t *v_out_dev, int *err_dev, void *stream);

/* Most requests of one w12_attend call. */
#define W12_ATTEND_MAX_R 512

/* Bytes of workspace w12_attend needs (0 on invalid arguments; max_len and
 * prefix_len as in the call).  A workspace serves calls of all sizes that
 * need no more than it has. */
size_t w12_attend_workspace_size(const w12_kv *kv, int64_t R, int64_t T, int q_heads, int64_t max_len,
                                 int64_t prefix_len);

/*
 * Causal attention of R * T new tokens over the cache (their own keys and
 * values are in it: w12_kv_append), grouped query heads:
 *   out[n, h] = sum_j softmax_j(scale q[n, h] . k[j, h / G]) v[j, h / G],
 *   G = q_heads / kv->heads, over the keys j <= position of token n.
 *   q_dev: bf16, token n's heads at q_dev + n * q_stride; 16-byte aligned,
 *     q_stride a multiple of 8.
 *   out_dev: bf16, token stride out_stride (a multiple of 4), 8-byte aligned,
 *     not overlapping the inputs.
 *   lse_dev: NULL, or fp32 [R * T][q_heads]: log(sum_j exp(scale q . k_j)).
 *   max_len: no kv_len is above it (a longer one records W12_ERR_DEVICE and
 *     is cut there); it only bounds the work.  At most 2^31 - 256.
 *   prefix_len: 0, or the number of leading keys that all requests with keys
 *     share (the same rows of the cache, or copies): as far as they fill tiles
 *     of 128 keys that every token of these requests sees, they are read once
 *     for the whole batch, through the first such request's row of the table.
 *     Each such request's row names all of its pages, the prefix's among
 *     them.  Not tied to page boundaries.  A request with kv_len <= 0 (an
 *     idle slot) takes no part: its row and its queries may hold anything.
 * A token that sees no key (a padding token, kv_len = 0) gives zeros and
 * lse = -infinity.  Keys past a token's position, rows past kv_len and pages
 * not named by the table never reach a result, whatever they hold.  Scores,
 * the running maximum and sums are fp32; the weights of the second product
 * are rounded to bf16 (bf16 cache) or, times their value's scale, to fp16
 * (e4m3 cache; fp16 ends at 2^-24, so a weight times its scale is kept down to
 * 2^-31 of the row's largest weight times the largest value scale it sees).
 * The order of every sum is fixed by the arguments, the lengths and the GPU's
 * SM count, so repeated calls give identical bits.  head_dim 64 or 128; 1 <= R
 * <= W12_ATTEND_MAX_R; q_heads a multiple of kv->heads.
 * Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_WORKSPACE,
 * W12_ERR_CUDA.  Device errors in word 0 of ws: W12_ERR_DEVICE (a length
 * above max_len or the table, a page outside the cache, which reads as page
 * 0), W12_ERR_TIMEOUT.
 */
int w12_attend(const w12_kv *kv, const uint16_t *q_dev, int64_t q_stride, int64_t R, int64_t T, int q_heads,
               const int32_t *block_table_dev, int64_t blocks, const int32_t *kv_len_dev, int64_t max_len,
               int64_t prefix_len, float scale, uint16_t *out_dev, int64_t out_stride, float *lse_dev, void *ws_dev,
               size_t ws_bytes, void *stream);

/* Largest V of w12_sample. */
#define W12_SAMPLE_MAX_V 524288

/* Bytes of workspace w12_sample needs (0 on invalid arguments). */
size_t w12_sample_workspace_size(int64_t R, int64_t T, int64_t V);

/*
 * Sample one token for each of R * T rows of logits from given random
 * numbers, and accept drafts against the sampled tokens.
 *   logits_dev: [R*T][V] row-major, dtype W12_F32 or W12_BF16 (4- or 2-byte
 *     aligned; 16-byte aligned rows are read faster).
 *   temperature_dev, top_k_dev, top_p_dev, min_p_dev: [R] per request (fp32,
 *     top_k int32), each may be NULL (temperature 1; no cut).
 *   u_dev: [R*T] fp32 in [0, 1), one random number per row (24 bits count).
 * Per row, with max its largest logit and t the temperature:
 *   w_i = round(2^31 e^((x_i - max) / t)), tokens ordered by logit, equal ones
 *   by index; a NaN counts as -infinity (never sampled).
 *   top_k (0 < top_k < V): the first top_k tokens stay.
 *   top_p (< 1): of those, a token stays while the weight before it is less
 *     than top_p (in units of 2^-24) times their whole weight; the first always.
 *   min_p (> 0): of those, tokens with w_i >= min_p 2^31 stay.
 *   tokens_dev[row] = the first index, in index order, at which the sum of the
 *     staying weights W passes u W; prob_dev[row] (may be NULL) = its w / W.
 *   t <= 0 (or NaN): the lowest index of the largest logit, probability 1.
 *   (0 < t < 2^-128, where 1 / t is no fp32 number, counts as 2^-128.)
 *   A row without a logit above -infinity, or whose tokens min_p > 1 all
 *   removes: token -1, probability 0.
 * The sums are whole numbers, so a result does not depend on how a row is
 * cut over the GPU.
 * Acceptance (accept_len_dev NULL: none), the rule of w12_verify_greedy on
 * the sampled tokens: accept_len[r] = first i < T - 1 with draft[r, i] !=
 * tokens[r, i], else T - 1; next_tok[r] = tokens[r, accept_len[r]]: every
 * committed token is the target model's own sample.
 *   draft_dev: [R][T-1] int32 (may be NULL when T == 1).
 * R >= 1, T >= 1, R * T < 2^27, 1 <= V <= W12_SAMPLE_MAX_V.
 * Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_WORKSPACE,
 * W12_ERR_CUDA.
 */
int w12_sample(const void *logits_dev, int dtype, int64_t R, int64_t T, int64_t V, const float *temperature_dev,
               const int32_t *top_k_dev, const float *top_p_dev, const float *min_p_dev, const float *u_dev,
               int32_t *tokens_dev, float *prob_dev, const int32_t *draft_dev, int32_t *accept_len_dev,
               int32_t *next_tok_dev, void *ws_dev, size_t ws_bytes, void *stream);

/* --------------------------------------------------------------------- */
/* Around a draft model                                                  */
/* --------------------------------------------------------------------- */

/*
 * The calls from here on serve the other half of speculative decoding, the
 * draft model: the addition and norm between two products of either model,
 * products with 4-bit weights (a drafter's weights may lose bits, the
 * target's verification makes up for them), and the verification of sampled
 * drafts.  The SpecPilot pages describe none of them; they are this
 * library's own.  They use programmatic dependent launch as the decode-step
 * calls do (packing, encoding and decoding do not).
 */

/* Largest row of w12_add_norm. */
#define W12_NORM_MAX_DIM 32768

/*
 * Residual addition and root-mean-square norm of `rows` rows of `dim`:
 *   h = x + delta,  y = h (weight + offset) / sqrt(mean(h^2) + eps).
 *   x_dev: x_dtype W12_F32 or W12_BF16; delta_dev (NULL: none): delta_dtype
 *     the same two; row r at x_dev + r * x_stride (elements; any stride).
 *   weight_dev: [dim] W12_F32 or W12_BF16, NULL: ones.  offset: 0, or 1 for
 *     models that store weight - 1.
 *   residual_dev (may be NULL): h in x's type, rounded once; the norm is of
 *     the unrounded h.  It may be x_dev itself with x's stride, or, where the
 *     types agree, delta_dev with delta's.
 *   out_dev: out_dtype W12_BF16, or W12_E4M3 with scale_dev [rows] fp32 (for
 *     W12_BF16 NULL): scale = amax / 448 of the row's y, codes round(y * (448
 *     / amax)) (nearest even); a row whose amax is at most 1e-30 is stored as
 *     zeros with scale 0, one that holds a NaN or an infinity as zeros with
 *     scale NaN.  Rows of out_dev and residual_dev at their strides, at least
 *     dim apart.
 * Pointers are aligned to their elements; rows that start on 16-byte
 * boundaries with dim a multiple of 8 are read faster.  Other than named,
 * outputs overlap nothing.  Sums are fp32, in a fixed order, of the row scaled
 * by a power of two where its squares would pass fp32's ends; |h (weight +
 * offset)| is to stay below 3.4e38 for a row to be finite, and |weight + offset|
 * below 2^120 where the mean of h^2 is below 2^-100.  A row of zeros with eps 0
 * gives zeros.
 * 1 <= dim <= W12_NORM_MAX_DIM, 0 <= rows < 2^31, eps >= 0 and finite.
 * Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_CUDA.
 */
int w12_add_norm(const void *x_dev, int64_t x_stride, int x_dtype, const void *delta_dev, int64_t delta_stride,
                 int delta_dtype, const void *weight_dev, int weight_dtype, float offset, float eps, int64_t rows,
                 int64_t dim, void *residual_dev, int64_t residual_stride, void *out_dev, int64_t out_stride,
                 int out_dtype, float *scale_dev, void *stream);

/*
 * 4-bit weights.  A K x N matrix (a linear layer's [N][K]) of e2m1 codes with
 * an e4m3 scale for 16 consecutive k of a column and one fp32 number:
 *   W[k, n] = code[n, k] scales[n, k / 16] scale,
 * codes 0, 0.5, 1, 1.5, 2, 3, 4, 6 (bits 2-0) with bit 3 as the sign.  The
 * plain form has codes [N][K / 2] bytes, the even k in a byte's low four bits,
 * and scales [N][K / 16] bytes.  The products read a blob: for tile t of 256
 * columns and group kg of 128 k, unit t * K / 128 + kg is a block of
 * W12_FP4_UNIT_BYTES:
 *   [0, 16384)      codes: column c's 64 bytes at 64 c, four 16-byte chunks of
 *                   four 32-bit words; chunk j at j ^ ((c >> 1) & 3), its word q
 *                   holds k = 64 (q >> 1) + 16 j + 8 (q & 1) .. + 7: the even k in
 *                   the low half, the odd ones in the high half; of a half's
 *                   codes 0 .. 3 the magnitudes at bits 8-6, 5-3, 2-0, 11-9, the
 *                   signs at 15, 12, 14, 13
 *   [16384, 18432)  scales: column c's 8 at 16384 + 8 c, that of k / 16 = g at
 *                   2 (g & 3) + (g >> 2): 5 exponent bits (bias 9), 3 mantissa
 *                   bits, no sign (a negative scale turns the codes' signs); a
 *                   zero scale is 0 with zero codes, NaN is 0xAF
 * Columns past N are zeros.  K is a multiple of 128.
 */
#define W12_FP4_UNIT_BYTES 18432
typedef struct w12_fp4 {
    const void *blob; /* w12_fp4_bytes(K, N) bytes on the device, 256-byte aligned */
    int64_t K, N;
    float scale;      /* in [2^-100, 2^100] */
    int32_t reserved; /* 0 */
} w12_fp4;

/* Bytes of a blob (0 for a shape that is not served). */
size_t w12_fp4_bytes(int64_t K, int64_t N);

/* The blob of a matrix in the plain form (codes_dev 16-byte, scales_dev
 * 8-byte aligned).  Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN,
 * W12_ERR_CUDA. */
int w12_fp4_pack(const uint8_t *codes_dev, const uint8_t *scales_dev, int64_t K, int64_t N, void *blob_dev, void *stream);

/*
 * The blob of a bf16 matrix w_dev [N][K] (16-byte aligned) for a given scale
 * (usually the largest |w| / 2688, which uses the whole range), in fp32: per 16 k
 * s = the e4m3 number nearest to max |w| / (6 scale), at least 2^-9 where a weight
 * is not 0, and the codes nearest to |w| (1 / (s scale)), ties to even (of the
 * rounded product: where |w| lies within 2^-22 of the middle between two codes it
 * may be either).  Weights past the range take the largest code; a NaN turns its
 * 16 weights into NaN.
 * Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_CUDA.
 */
int w12_fp4_encode(const uint16_t *w_dev, int64_t K, int64_t N, float scale, void *blob_dev, void *stream);

/* The weights back as fp32 [N][K] (16-byte aligned).  Errors as above. */
int w12_fp4_decode(const w12_fp4 *w, float *out_dev, void *stream);

/* Bytes of workspace w12_fp4_gemm (count 1) and w12_fp4_gemm_batched need for
 * these matrices and M (0 on invalid arguments); blob and scale are not read.  A
 * workspace serves calls of all sizes that need no more than it has. */
size_t w12_fp4_gemm_workspace_size(const w12_fp4 *w, int count, int64_t M);

/*
 * y[m, n] = sum_k x[m, k] W[k, n], 1 <= M <= W12_MAX_M.
 *   x_dev: [M][K] x_dtype W12_BF16 or W12_E4M3, 16-byte aligned; for W12_E4M3
 *     x_scale_dev [M] fp32 (w12_add_norm writes both), else NULL.
 *   y_dev: [M][N] y_dtype W12_F32 or W12_BF16, not overlapping the inputs.
 *   options: 0 or W12_OPT_EARLY_WEIGHTS (as in w12_gemm_ex: the blob was not
 *     written by the kernel launched just before).
 * code times the group's scale is exact in the products' type; sums are fp32,
 * in an order fixed by the shapes, M and the GPU's SM count, so repeated
 * calls give identical bits.  From 17 tokens on they are the tensor core's own
 * sums over up to 8192 k, whose additions are cut, not rounded: a sum of one
 * sign comes out low by up to 7e-6 of itself, whatever K.
 * Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_WORKSPACE,
 * W12_ERR_CUDA.  Device errors in word 0 of ws: W12_ERR_TIMEOUT.
 */
int w12_fp4_gemm(const w12_fp4 *w, const void *x_dev, int x_dtype, const float *x_scale_dev, int64_t M, void *y_dev,
                 int y_dtype, void *ws_dev, size_t ws_bytes, int options, void *stream);

/* count independent products (1 <= count <= W12_MAX_BATCH) of one M in one
 * launch, as w12_gemm_batched: host arrays of count matrices and device
 * pointers (x_scale_dev NULL for W12_BF16). */
int w12_fp4_gemm_batched(const w12_fp4 *w, const void *const *x_dev, int x_dtype, const float *const *x_scale_dev, int64_t M,
                         void *const *y_dev, int y_dtype, int count, void *ws_dev, size_t ws_bytes, int options,
                         void *stream);

/* Cuts of a distribution per request, as in w12_sample: [R] each, or NULL
 * (temperature 1; no cut). */
typedef struct w12_cut {
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p;
} w12_cut;

/* Bytes of workspace w12_verify_sampled needs (0 on invalid arguments).  A
 * workspace serves calls of all sizes that need no more than it has. */
size_t w12_verify_sampled_workspace_size(int64_t R, int64_t T, int64_t V);

/*
 * Verify R sampled draft blocks against the target's probabilities, from given
 * random numbers (the greedy rule is w12_verify_greedy; w12_sample accepts
 * drafts that equal the target's own samples, this accepts more of them when
 * they were sampled from a distribution near the target's).
 *   logits_dev: [R*T][V] of the target, dtype W12_F32 or W12_BF16: row i of a
 *     block is its prediction after [last token, d0 .. d(i-1)].
 *   draft_logits_dev: [R*(T-1)][V] of the drafter, draft_dtype: row i is what
 *     draft token i was drawn from.  Both aligned to their elements; 16-byte
 *     aligned rows are read faster.
 *   draft_dev: [R][T-1] int32; a token outside [0, V) is none: the block ends
 *     there.  (These three may be NULL when T == 1.)
 *   target_cut, draft_cut (may be NULL): what p and q are the distributions of
 *     -- w / W of the tokens that stay, with w12_sample's weights and rules
 *     (temperature <= 0: its one token); draft_cut is the one the drafts were
 *     drawn with.
 *   u_dev: [R][T] fp32 in [0, 1): u[r, i < T-1] for draft i, u[r, T-1] for the
 *     next token.
 * With p and q in fp32 (a weight times the rounded 1 / W):
 *   accept_len_dev[r] = first i < T-1 without u[r, i] q_i(d_i) < p_i(d_i), else
 *     T-1 =: n;
 *   next_tok_dev[r] = the first index at which the sum of the weights passes
 *     u[r, T-1] times their whole sum: for n < T-1 (with a draft there) the
 *     weights round(2^44 max(p_n - q_n, 0)), where they are not all 0, else the
 *     target's own (the token that w12_sample draws).  -1: no token of the row
 *     stays.
 *   ratio_dev (may be NULL): [R][T-1] fp32, min(1, p / q) of every draft (0
 *     where p is 0 or there is no draft).
 * R >= 1, T >= 1, R * T < 2^26, 1 <= V <= W12_SAMPLE_MAX_V.  Sums are whole
 * numbers: repeated calls give identical results.
 * Errors: W12_ERR_ARG, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_WORKSPACE,
 * W12_ERR_CUDA.  Device errors in word 0 of ws: W12_ERR_TIMEOUT.
 */
int w12_verify_sampled(const void *logits_dev, int dtype, const void *draft_logits_dev, int draft_dtype, int64_t R,
                       int64_t T, int64_t V, const int32_t *draft_dev, const w12_cut *target_cut,
                       const w12_cut *draft_cut, const float *u_dev, float *ratio_dev, int32_t *accept_len_dev,
                       int32_t *next_tok_dev, void *ws_dev, size_t ws_bytes, void *stream);

/*
 * Read (and clear) the sticky device error word of a workspace: waits for
 * `stream`, copies word 0 to *err_host, then zeroes it.  Returns W12_OK or
 * W12_ERR_CUDA.  *err_host is W12_OK or the first error recorded since the
 * word was last cleared: W12_ERR_DEVICE (a kernel met an escape index
 * outside the escape list) or W12_ERR_TIMEOUT (a bounded wait ran out; the
 * call's outputs are undefined).
 */
int w12_get_device_error(void *ws_dev, int *err_host, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* W12_H */
