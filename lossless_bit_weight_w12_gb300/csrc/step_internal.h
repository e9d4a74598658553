// step_internal.h -- declarations shared by the decode-step calls (paged
// key/value cache, attention over it, sampling): argument blocks of the
// kernels and their launchers.  Not installed.
#pragma once

#include <cuda.h>

#include <cstddef>
#include <cstdint>

#include "../../include/w12.h"
#include "w12_internal.h"

namespace w12 {

// Launch with programmatic stream serialization (the kernel's CTAs may start
// while the previous kernel of the stream drains; they call pdl_wait()
// before their first access to global memory).
#ifdef __CUDACC__
template <typename Args>
int launch_step(void (*kernel)(Args), int grid, int threads, size_t smem, int cluster, void *stream, const Args &a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = unsigned(cluster);
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? W12_OK : W12_ERR_CUDA;
}
#endif

struct AppendArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, out_stride;  // elements per token
    uint16_t *q_out;
    void *kc, *vc;
    float *ks, *vs;
    const int32_t *table, *kv_len;
    const float *rope;
    int64_t rope_positions, tokens, table_cols, n_pages;
    int32_t T, q_heads, heads, page, page_log2, rot, interleaved;
    int32_t parts;  // groups of lanes per token
    int *err;
};
int launch_append(const AppendArgs &a, int x_dtype, int head_dim, int kv_dtype, int sms, void *stream);

struct ReadArgs {
    const void *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *cu_len;
    uint16_t *k_out, *v_out;
    int64_t R, tokens, table_cols, n_pages;
    int32_t heads, page, page_log2;
    int *err;
};
int launch_read(const ReadArgs &a, int head_dim, int kv_dtype, int sms, void *stream);

// Attention (kernels_attend.cu, kernels_attend_tc.cu); the work split is
// described in attend_device.cuh.
constexpr int kAttTile = 64;     // keys per tile of the register kernel
constexpr int kAttTcTile = 128;  // of the tensor-memory kernel

// One launch's share of the work: units, their tiles on a line, the CTAs
// that cut it, and where the segments' results go.
struct AttendLine {
    int32_t pu, su;   // units per head: row blocks of all requests under the prefix, row blocks per request
    int32_t rt;       // query rows per unit
    int32_t halves;   // results per segment (2: its tiles in two alternating halves)
    int32_t grid;     // its workers (CTAs, or halves of CTAs) at most; 0: the line is not used
    float *part_o;    // [slots][halves][head_dim][rt]; the register kernel's: [slots][rt][head_dim]
    float2 *part_ml;  // [slots][halves][rt]: reference exponent (log2 units) and sum
};

// Lines: the tensor-memory kernel on the prefix; what follows, request by
// request, in the tensor-memory kernel or in the register kernel.
enum { kLinePrefix = 0, kLineRequests = 1, kLineRest = 2, kLines = 3 };

struct AttendArgs {
    CUtensorMap mk, mv;  // the cache as rows of head_dim channels; boxes of min(page, 64) rows
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    const float *ks, *vs;
    const int32_t *table, *kv_len;
    int64_t q_stride, out_stride;
    int64_t n_pages, table_cols;
    int32_t R, T, G, heads, page, page_log2;
    int32_t rows;      // R * T * G query rows per key head
    int32_t prefix, max_len;
    int32_t self;      // the line of this launch
    int32_t sms;
    float scale_log2;  // scale * log2(e)
    int *err;
    uint64_t per_g;     // 2^64 / G, rounded up (G = 1: not used)
    uint32_t *arrived;  // [workers] segments of a unit that are done; zero between calls
    int32_t *plan;      // for the join: W, both lines' workers, the R + 1 cumulative tiles of the requests
    int32_t join;       // 1: a join kernel adds up the results
    int32_t split;      // its warps per row group and channels: 1, 2, 4 or 8
    AttendLine line[kLines];
};
int attend_make_maps(AttendArgs &a, const w12_kv *kv);
int launch_attend_rest(const AttendArgs &a, int head_dim, int kv_dtype, void *stream);
int launch_attend_tc(const AttendArgs &a, int head_dim, int kv_dtype, void *stream);
int launch_attend_join(const AttendArgs &a, int head_dim, void *stream);

struct SampleArgs {
    const void *logits;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t *top_k, *draft;
    int32_t *tokens, *accept_len, *next_tok;
    float *prob;
    uint32_t *counter;
    int64_t V, rows, R, T;
    int32_t chunk;      // logits per CTA of a row's cluster
    int32_t resident;   // the chunk fits in shared memory
    int32_t keep_w;     // and so do its weights
    int32_t vec;        // 16-byte loads: every chunk starts on a 16-byte boundary
};
int launch_sample(SampleArgs &a, int dtype, void *stream);

}  // namespace w12
