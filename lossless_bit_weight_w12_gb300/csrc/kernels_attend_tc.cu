// kernels_attend_tc.cu -- attention on the tensor cores (tcgen05), for parts
// with many query rows per key head: the prefix that all requests share,
// draft blocks.  The mathematics is kernels_attend.cu's.
//
// A CTA has two slots, each a block of 128 query rows with its own region of
// tensor memory -- scores S (128 columns; the weights P take their place) and
// output O (head_dim columns) -- and its own four softmax warps (thread = row =
// tensor-memory lane).  Units of 256 rows: slot s has rows
// 128 s .., both use every tile.  Units of 128 rows: the slots take alternate
// tiles, and their results are added up at the end.  Per tile of 128 keys
// and slot:
//   S = Q K^T      A = the queries in shared memory, B = the keys as they lie
//                  in the ring (K-major, 128-byte swizzle)
//   softmax        S to registers, maximum, exponentials, P back
//   O += P V       A = P from tensor memory, B = the values as they lie in
//                  the ring (the channels contiguous)
// While one slot's warps work on S the tensor cores work for the other.  128
// keys a tile, because a product of N = 64 takes nearly as long as one of N =
// 128 (about 45 and 64 cycles), and because every hand-over between the warps
// and the tensor cores costs some 300 cycles (in halves of 64 keys, a slot's
// next scores ready during its softmax: 77 us against 54 for 8 requests x 16
// tokens, 105 against 98 under a prefix).  The issuing thread orders the
// products of its slot: S of tile i + 1 overwrites P of tile i after the
// product that reads it.  Keys and values are separate stages of the ring:
// the keys' is free as soon as S is there.
//
// O stays in tensor memory.  It is rescaled only when the maximum has grown
// by more than 2^8 since the last time (the exponentials are then at most
// 2^8, or, e4m3, 2^15 after the value's scale: inside fp16), by the slot's
// own warps, between two products.
//
// e4m3 tiles pass four converter warps, which write them as fp16 tiles in
// the same layout into a second ring.
//
// Tiles with keys that some row must not see (a draft block's own tokens, the
// end of the keys) have their scores masked in the registers.  A weight of 0
// does not keep out a value that is not finite, so value rows past the end
// are set to zero before the product, and channels that are not finite in
// rows that only some query rows see are taken out and added by hand.  (The
// same for weights whose value scale is not finite.)
//
// What bounds it: a slot's chain of scores, softmax and product, about 6500
// cycles for two tiles on e4m3 (the multiplications by the scales) and 3300 on
// bf16, where the products alone take 2048.  8 requests x 16 tokens of 700 ..
// 9000 keys, 8 key heads: e4m3 (82 MB) 51 us and bf16 (160 MB) 49, each with 9
// for the join; the prefix of 16000 for 128 requests of 48 heads: 79 us on 90
// SMs, 50 GFLOP.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "attend_device.cuh"
#include "device_common.cuh"
#include "tcgen05_common.cuh"

namespace w12 {

namespace {

constexpr float kNegInf = -INFINITY;
constexpr int kProdWarp = 8;   // 8, 11: copies of keys, values
constexpr int kIssueWarp = 9;  // 9, 10: products of slot 0, 1 (9 owns the tensor memory)
constexpr int kConvWarp = 12;  // 12 .. 15: e4m3 to fp16
constexpr uint32_t kTmem = 512, kSlotCols = 256, kOCol = 128;
constexpr int kKT = kAttTcTile;

template <int D, bool Q8, bool TWO>
struct TC {
    static constexpr int kThreads = Q8 ? 512 : 384;
    // The softmax warps need the registers that the others do not: shares of
    // the launch's 12 x 168 or 16 x 128 per lane.
    static constexpr int kRegsSoftmax = Q8 ? 184 : 216, kRegsOther = 72;
    static constexpr int kLaunchRegs = Q8 ? 16 * 128 : 12 * 168;
    static_assert(8 * kRegsSoftmax + (kThreads / 32 - 8) * kRegsOther <= kLaunchRegs, "register shares");
    static constexpr int kHalf = kKT * D * 2;           // keys, or values, of a tile as operands
    static constexpr int kQ = (TWO ? 256 : 128) * D * 2;
    static constexpr int kInScale = kKT * D;            // e4m3 input stage: codes, then 128 scales
    static constexpr int kIn = Q8 ? kKT * D + 1024 : kHalf;
    static constexpr int kScales = kKT + 4;             // floats per half tile: scales, and (values) their bound
    // The keys' stage is free before the softmax has read their scales, and
    // the values' scales are given out before their stage; a half tile's
    // scales are written over 8 halves (4 tiles) later, which the converters
    // reach only after a product that follows this tile's softmax.
    static constexpr int kScaleRing = 8;
    static constexpr int kFixed = (int(sizeof(AttShared)) + 15) / 16 * 16 + 1024 + (Q8 ? kScaleRing * kScales * 4 + 1024 : 0);
    static constexpr int kRoom = 227 * 1024 - kFixed - kQ;
    // Operand stages.  With units of 128 rows the values' stages (bf16: the
    // keys', too) have to stay with one slot: a multiple of 4 in turn, or,
    // e4m3, one for the keys and one per slot for the values.  e4m3 leaves
    // room for the input ring, whose stages each belong to the keys or to the
    // values (an even number) where these have converters of their own.
    static constexpr bool kOwn = Q8 && !TWO;
    static constexpr int kOpFit = (Q8 ? kRoom - 3 * kIn : kRoom) / kHalf;
    static constexpr int SO = kOwn ? 3 : TWO ? (kOpFit > 4 && Q8 ? 4 : kOpFit > 8 ? 8 : kOpFit) : kOpFit >= 8 ? 8 : 4;
    static constexpr int kInFit = (kRoom - SO * kHalf) / kIn;
    static constexpr int SI = Q8 ? (kInFit > 8 ? 8 : kOwn ? kInFit / 2 * 2 : kInFit) : SO;
    static constexpr int kRing = Q8 ? SI * kIn + SO * kHalf : SO * kHalf;
    static constexpr size_t kSmem = size_t(kQ) + kRing + kFixed;
    static_assert(SO >= 3 && SI >= 3 && SO <= 8 && (!Q8 || SO + 1 < kScaleRing) && (TWO || kOwn || SO % 4 == 0) && (!kOwn || SI % 2 == 0) && kSmem <= 227 * 1024, "shared memory");
    static_assert((4 * 8 + 13 + kScaleRing / 2) * 8 + 32 <= 1008, "barriers");
};

template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ void tmem_load1(uint32_t taddr, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r)
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_store1(uint32_t taddr, uint32_t r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// f(c, columns 64 c .. of this lane's row) for c < 2.
template <typename F>
__device__ __forceinline__ void by_columns(uint32_t ts, F f) {
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
        float2 x[32];
        tmem_load32(ts + 64u * uint32_t(c), reinterpret_cast<uint32_t *>(x));
        tmem_load32(ts + 64u * uint32_t(c) + 32u, reinterpret_cast<uint32_t *>(x + 16));
        tmem_wait_ld();
        tmem_landed32(reinterpret_cast<uint32_t *>(x));
        tmem_landed32(reinterpret_cast<uint32_t *>(x + 16));
        f(c, x);
    }
}

// Barriers of a part of the softmax warps; any of them: x.
__device__ __forceinline__ bool bar_any(int id, int threads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(x)), "r"(id), "r"(threads)
        : "memory");
    return r != 0u;
}

// 16-byte piece c of row `key` of a tile's values in an operand stage.
__device__ __forceinline__ uint32_t value_at(uint32_t stage, int key, int c) {
    return stage + uint32_t((c >> 3) * kKT * 128 + key * 128 + (((c & 7) ^ (key & 7)) << 4));
}

// Bits of the exponent of fp16, bf16: all ones where a number is not finite.
template <bool Q8>
__device__ __forceinline__ bool odd16(uint32_t x) {
    constexpr uint32_t e = Q8 ? 0x7C00u : 0x7F80u;
    return (x & e) == e;
}
template <bool Q8>
__device__ __forceinline__ bool odd_piece(const uint4 &x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) odd = odd || odd16<Q8>(w[j]) || odd16<Q8>(w[j] >> 16);
    return odd;
}

// Adds the channels that are not finite in the values' rows from..to - 1 to
// the outputs of the rows that see them (row r of the tile: r <= seen), with
// the weights as they are in tensor memory.
template <int D, bool Q8>
__device__ __noinline__ void add_odd(uint32_t stage, int from, int to, int seen, uint32_t t_p, uint32_t t_o) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int r = from; r < to; ++r) {
        uint32_t pieces = __ballot_sync(0xFFFFFFFFu, lane < D / 8 && odd_piece<Q8>(lds128(value_at(stage, r, lane % (D / 8)))));
        if (!pieces) continue;
        uint32_t pp;
        tmem_load1(t_p + uint32_t(r >> 1), pp);
        const uint16_t ph = uint16_t(r & 1 ? pp >> 16 : pp);
        const float w = Q8 ? __half2float(__ushort_as_half(ph)) : bf16_bits_to_float(ph);
#pragma unroll 1
        for (; pieces; pieces &= pieces - 1) {
            const int c = __ffs(pieces) - 1;
            const uint4 x = lds128(value_at(stage, r, c));
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint16_t h = uint16_t(e & 1 ? xs[e >> 1] >> 16 : xs[e >> 1]);
                if (!odd16<Q8>(h)) continue;  // (the same for all lanes)
                const float v = Q8 ? __half2float(__ushort_as_half(h)) : bf16_bits_to_float(h);
                uint32_t o;
                tmem_load1(t_o + uint32_t(8 * c + e), o);
                if (r <= seen) o = __float_as_uint(__uint_as_float(o) + w * v);
                tmem_store1(t_o + uint32_t(8 * c + e), o);
                tmem_wait_st();
            }
        }
    }
}

// e4m3: a key's weight is zero for the rows that must not see it, whatever
// its value's scale holds (0 times a scale that is not finite is NaN).
__device__ __noinline__ void clear_weights(const float *vsc, int from, int to, int seen, uint32_t t_p) {
#pragma unroll 1
    for (int r = from; r < to; ++r) {
        if (fabsf(vsc[r]) <= 3.0e38f) continue;
        uint32_t w;
        tmem_load1(t_p + uint32_t(r >> 1), w);
        if (r > seen) w &= r & 1 ? 0xFFFFu : 0xFFFF0000u;
        tmem_store1(t_p + uint32_t(r >> 1), w);
        tmem_wait_st();
    }
}

// e4m3: as `lift`, which the converters make of all value scales of a tile, but
// of those that the lane's row sees (r <= seen; before `from`: all rows), so
// that a later token's do not reach it.  It is the same, as a rule, for all rows.
// vsc: where the scales are.
__device__ __noinline__ float seen_lift(uint32_t vsc, float lift, int from, int until, int seen) {
    const auto bits = [](uint32_t x) { return __uint_as_float(x) <= 3.0e38f ? x : 0u; };
    const int mine = 4 * int(threadIdx.x & 31);
    const uint4 y = lds128(vsc + 4u * uint32_t(mine));
    uint32_t top = max(max(mine < from ? bits(y.x) : 0u, mine + 1 < from ? bits(y.y) : 0u),
                       max(mine + 2 < from ? bits(y.z) : 0u, mine + 3 < from ? bits(y.w) : 0u));
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (exp_above(__uint_as_float(top)) - 7.0f == lift) return lift;
#pragma unroll 1
    for (int r = from; r < until; ++r) {
        const uint32_t x = bits(lds32(vsc + 4u * uint32_t(r)));
        if (r <= seen) top = max(top, x);
    }
    return exp_above(__uint_as_float(top)) - 7.0f;
}

// Zeros in their place; part `me` of n of the work.
template <int D, bool Q8>
__device__ __noinline__ void clear_odd(uint32_t stage, int from, int to, int me, int n) {
    for (int x = me; x < (to - from) * (D / 8); x += n) {
        const uint32_t at = value_at(stage, from + x / (D / 8), x % (D / 8));
        const uint4 y = lds128(at);
        if (!odd_piece<Q8>(y)) continue;
        uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] &= (odd16<Q8>(w[j]) ? 0xFFFF0000u : ~0u) & (odd16<Q8>(w[j] >> 16) ? 0xFFFFu : ~0u);
        sts128(at, w[0], w[1], w[2], w[3]);
    }
}

template <int D, bool Q8, bool TWO>
__global__ void __launch_bounds__(Q8 ? 512 : 384, 1) attend_tc_kernel(const __grid_constant__ AttendArgs a) {
    using C = TC<D, Q8, TWO>;
    constexpr int SO = C::SO, SI = C::SI, KS = D / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    const uint32_t ring = base + uint32_t(C::kQ);                    // input ring (e4m3), operand ring
    const uint32_t ops = ring + uint32_t(Q8 ? SI * C::kIn : 0);
    unsigned char *fixed = smem + C::kQ + C::kRing;
    AttShared &sh = *reinterpret_cast<AttShared *>(fixed);
    unsigned char *misc = fixed + (sizeof(AttShared) + 15) / 16 * 16;
    uint64_t *in_full = reinterpret_cast<uint64_t *>(misc), *in_empty = in_full + SI;
    uint64_t *op_full = Q8 ? in_empty + SI : in_full, *op_empty = Q8 ? op_full + SO + 1 : in_empty;
    uint64_t *s_full = (Q8 ? op_empty + SO : in_empty + SI), *p_full = s_full + 2, *q_full = s_full + 4,
             *o_done = s_full + 6, *fin = s_full + 8, *token = s_full + 10, *vs_full = s_full + 12;
    WaitCtl &ctl = *reinterpret_cast<WaitCtl *>(s_full + 12 + C::kScaleRing / 2);
    uint32_t &s_tmem = *reinterpret_cast<uint32_t *>(reinterpret_cast<unsigned char *>(&ctl) + sizeof(WaitCtl));
    float *scales = reinterpret_cast<float *>(misc + 1024);          // [kScaleRing][128 scales, their bound]
    float *q_up = scales + (Q8 ? C::kScaleRing * C::kScales : 0);    // e4m3: [256] powers of two of the query rows
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (base & 1023u) {  // the swizzled boxes and operands need 1024-byte aligned stages
        if (threadIdx.x == 0) record_error(a.err, W12_ERR_DEVICE);
        return;
    }
    if (threadIdx.x == 0) {
        constexpr uint32_t kUsers = TWO ? 2 : 1;       // slots that use a stage
        constexpr uint32_t kConverters = TWO ? 4 : 2;  // warps that write an operand stage
        for (int s = 0; s < SI; ++s) {
            mbar_init(&in_full[s], 1);
            mbar_init(&in_empty[s], Q8 ? kConverters : kUsers);
        }
        if (Q8)
            for (int s = 0; s < SO; ++s) {
                mbar_init(&op_full[s], kConverters);
                mbar_init(&op_empty[s], kUsers);
            }
        if (C::kOwn) mbar_init(&op_full[3], kConverters);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
            mbar_init(&q_full[s], 4);
            mbar_init(&o_done[s], 1);
            mbar_init(&fin[s], 1);
            mbar_init(&token[s], 1);
        }
        if (Q8)
            for (int s = 0; s < C::kScaleRing / 2; ++s) mbar_init(&vs_full[s], kConverters);
        ctl.abort = 0;
        ctl.limit_ns = kWaitLimitNs;
        mbar_fence_init();
    }
    if (warp == kIssueWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (lane == 0 && (warp == kProdWarp || warp == kProdWarp + 3)) prefetch_map(warp == kProdWarp ? &a.mk : &a.mv);
    att_start(a);
    const AttPlan plan = att_plan(a, sh, 1, 0);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = s_tmem;
    const AttendLine &ln = a.line[a.self];
    const int t0 = plan.t0, t1 = plan.t1;
    // the first of this slot's tiles from position k of a segment whose first
    // tile is the CTA's i0-th, and the step between them
    const auto first_tile = [](int i0, int slot) { return TWO ? 0 : (i0 & 1) != slot ? 1 : 0; };
    constexpr int kStep = TWO ? 1 : 2;

    // tile i's keys (kv = 0) or values (1): their operand stage, how often it
    // was used before
    const auto stage = [](int i, int kv) { return C::kOwn ? kv ? 1 + (i & 1) : 0 : (2 * i + kv) % SO; };
    const auto used = [](int i, int kv) { return C::kOwn ? kv ? i >> 1 : i : (2 * i + kv) / SO; };
    // Waits until it is filled.  One stage for all keys has a barrier per slot:
    // the slots wait for alternate tiles, and a slot that had not waited for
    // the tile before could take its phase for the next.
    const auto wait_operand = [&](int i, int kv) {
        if (C::kOwn)
            att_wait(&op_full[kv ? 1 + (i & 1) : 3 * (i & 1)], uint32_t(i >> 1) & 1u, &ctl, a.err);
        else
            att_wait(&op_full[stage(i, kv)], uint32_t(used(i, kv)) & 1u, &ctl, a.err);
    };
    // the roles, by warpgroup (a warpgroup changes its registers as one)
    if (warp < kProdWarp) {
        // ------------------------------------------------------- softmax
        regs_up<C::kRegsSoftmax>();
        const int slot = warp >> 2;
        const int row = 32 * (warp & 3) + lane;
        const uint32_t ts = tmem + uint32_t(slot) * kSlotCols + (uint32_t(32 * (warp & 3)) << 16);
        const uint32_t to = ts + kOCol;
        uint32_t n_s = 0, n_seg = 0;
        AttSeg seg = sh.first[0];
#pragma unroll 1
        for (int t = t0, n; t < t1; t += n) {
            if (t > t0) att_next(a, plan, sh, seg);
            const int i0 = t - t0, k0 = first_tile(i0, slot);
            n = min(seg.left, t1 - t);
            const size_t entry = size_t(seg.unit + int(blockIdx.x)) * size_t(ln.halves) + (TWO ? 0 : slot);
            const int in_unit = (TWO ? 128 * slot : 0) + row;
            const bool valid = in_unit < seg.nrows;
            const bool warp_valid = __any_sync(0xFFFFFFFFu, valid);
            const size_t at = entry * size_t(ln.rt) + in_unit;
            // ---- queries to shared memory, D / 8 lanes a row.  Units of 128
            // rows have one copy for both slots: their warps wait for one
            // another's products on the last one, then each copies half.
            float sc = fabsf(a.scale_log2);
            {
                constexpr int L = D / 8, RPW = 32 / L;            // lanes per row, rows per step of a warp
                constexpr int kRows = TWO ? 32 : 16;              // rows of this warp
                const int c = lane % L;
                const uint32_t qb = base + uint32_t(TWO ? slot : 0) * uint32_t(128 * D * 2);
                const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;  // scores grow with S
                const int first = TWO ? 32 * (warp & 3) : 16 * warp;
                constexpr int B = kRows / RPW;                    // loads in flight: all of them
                static_assert(kRows % RPW == 0, "rows of a warp");
                {
                    uint4 q[B];
                    int in_u = (TWO ? 128 * slot : 0) + first + lane / L;
                    int tok = att_token(a, seg.row0 + in_u), g = seg.row0 + in_u - tok * a.G;
                    const int step = att_token(a, RPW), step_g = RPW - step * a.G;
                    const uint16_t *src = a.q + int64_t(seg.head * a.G) * D + 8 * c;
#pragma unroll
                    for (int x = 0; x < B; ++x) {
                        q[x] = make_uint4(0, 0, 0, 0);
                        if (in_u < seg.nrows) q[x] = *reinterpret_cast<const uint4 *>(src + tok * a.q_stride + g * D);
                        in_u += RPW, tok += step, g += step_g;
                        if (g >= a.G) g -= a.G, ++tok;
                    }
                    if (!TWO) named_sync(256);
#pragma unroll
                    for (int x = 0; x < B; ++x) {
                        const int rq = first + x * RPW + lane / L;
                        uint32_t w[4] = {q[x].x, q[x].y, q[x].z, q[x].w};
                        if (Q8) {  // fp16, the row scaled by a power of two to below 2
                            uint32_t top = 0;
#pragma unroll
                            for (int y = 0; y < 4; ++y) top = max(top, max(w[y] & 0x7FFFu, (w[y] >> 16) & 0x7FFFu));
#pragma unroll
                            for (int o = L / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                            const int e = max(-100, min(126, int(top >> 7) - 127));
                            const float down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                w[y] = pack_f16(bf16_bits_to_float(w[y] & 0xFFFFu) * down,
                                                bf16_bits_to_float(w[y] >> 16) * down);
                            if (c == 0) q_up[(TWO ? 128 * slot : 0) + rq] = __uint_as_float(uint32_t(127 + e) << 23);
                        }
                        sts128(qb + uint32_t((c >> 3) * 128 * 128 + rq * 128) + uint32_t(((c & 7) ^ (rq & 7)) << 4),
                               w[0] ^ sign, w[1] ^ sign, w[2] ^ sign, w[3] ^ sign);
                    }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (TWO)
                __syncwarp();
            else
                named_sync(256);
            if (Q8) sc *= q_up[in_unit];
            sc = fmaxf(sc, 1e-37f);  // (a mask's -infinity times 0 would be NaN)
            const int all_see = att_seen_by_all(a, seg);
            const int pos = valid && a.self != kLinePrefix ? seg.key_end - a.T + att_token(a, seg.row0 + in_unit) - seg.req * a.T
                                                           : seg.key_end - 1;
            if (k0 >= n) {  // no tile of the segment is this slot's
                if (valid) ln.part_ml[at] = make_float2(kNegInf, 0.0f);
                continue;
            }
            if (seg.key + (k0 + 1) * kKT - 1 > all_see) {  // add_odd() may come before the first product
                const uint32_t zero[32] = {};
                for (int c = 0; c < D; c += 32) tmem_store32(to + uint32_t(c), zero);
                tmem_wait_st();
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[slot]);

            float m = kNegInf, l = 0.0f;
            for (int k = k0; k < n; k += kStep) {
                const int i = i0 + k;
                const int key0 = seg.key + k * kKT;
                const bool masked = key0 + kKT - 1 > all_see;
                // rows of the values that not every query row sees: from .. to - 1, then rows past the end
                const int from = masked ? max(all_see - key0 + 1, 0) : 0, until = max(min(seg.key_end - key0, kKT), from);
                const uint32_t vb = ops + uint32_t(stage(i, 1)) * uint32_t(C::kHalf);
                bool odd = false;
                // The scores come first, for every warp: their product was
                // issued after that of the slot's tile before, whose values it
                // had waited for, so the phase before of a values' stage (or
                // of its scales) is over and the parity below tells this one.
                // A warp that had not waited for those values would else take
                // their phase for this tile's, and touch a stage that is being
                // filled.
                att_wait(&s_full[slot], n_s++ & 1u, &ctl, a.err);
                tmem_fence_after();
                if (masked) {
                    wait_operand(i, 1);
                    const int x0 = TWO ? int(threadIdx.x) : row;
                    for (int x = from * (D / 8) + x0; x < until * (D / 8); x += TWO ? 256 : 128)
                        odd = odd || odd_piece<Q8>(lds128(value_at(vb, x / (D / 8), x % (D / 8))));
                    if (!Q8)  // (e4m3: the converters have done it)
                        for (int x = until * (D / 8) + x0; x < kKT * (D / 8); x += TWO ? 256 : 128)
                            sts128(value_at(vb, x / (D / 8), x % (D / 8)), 0u, 0u, 0u, 0u);
                    if (Q8 && row >= from && row < until)
                        odd = odd || !(fabsf(scales[(2 * i + 1) % C::kScaleRing * C::kScales + row]) <= 3.0e38f);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    odd = bar_any(TWO ? 1 : 2 + slot, TWO ? 256 : 128, odd);
                }
                if (warp_valid) {
                    float lift = 0.0f;
                    const uint32_t tk = smem_addr(scales + 2 * i % C::kScaleRing * C::kScales);
                    const uint32_t tv = tk + uint32_t(C::kScales) * 4u;  // (2 i + 1 is in the ring's same turn)
                    const int seen = pos - key0;
                    float top;
                    float2 xs[Q8 ? 1 : kKT / 2];
                    if (Q8) {
                        // Two passes over 64 columns at a time, by small loops
                        // (unrolled, the multiplications by the scales make
                        // the code miss the instruction cache: 73 us against 57
                        // for 8 x 16 tokens): the scaled scores go back to
                        // tensor memory.
                        float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
                        by_columns(ts, [&](int c, float2 (&x)[32]) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const uint4 z = lds128(tk + uint32_t(256 * c + 16 * j));
                                x[2 * j] = __fmul2_rn(x[2 * j], make_float2(__uint_as_float(z.x), __uint_as_float(z.y)));
                                x[2 * j + 1] =
                                    __fmul2_rn(x[2 * j + 1], make_float2(__uint_as_float(z.z), __uint_as_float(z.w)));
                            }
                            if (masked) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) {
                                    x[j].x = 64 * c + 2 * j <= seen ? x[j].x : kNegInf;
                                    x[j].y = 64 * c + 2 * j + 1 <= seen ? x[j].y : kNegInf;
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 32; ++j) mx[j & 3] = max3(mx[j & 3], x[j].x, x[j].y);
                            tmem_store32(ts + 64u * uint32_t(c), reinterpret_cast<const uint32_t *>(x));
                            tmem_store32(ts + 64u * uint32_t(c) + 32u, reinterpret_cast<const uint32_t *>(x + 16));
                        });
                        att_wait(&vs_full[i % (C::kScaleRing / 2)], uint32_t(i / (C::kScaleRing / 2)) & 1u, &ctl, a.err);
                        lift = __uint_as_float(lds32(tv + uint32_t(kKT) * 4u));
                        // keys that only some rows see (out of line: the loop
                        // has to stay in the instruction cache)
                        if (__builtin_expect(masked && from < until, 0)) lift = seen_lift(tv, lift, from, until, seen);
                        top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc + lift;
                        tmem_wait_st();
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_load32(ts + 32u * uint32_t(c), reinterpret_cast<uint32_t *>(xs + 16 * c));
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_landed32(reinterpret_cast<uint32_t *>(xs + 16 * c));
                        if (masked) {
#pragma unroll
                            for (int j = 0; j < kKT / 2; ++j) {
                                xs[j].x = 2 * j <= seen ? xs[j].x : kNegInf;
                                xs[j].y = 2 * j + 1 <= seen ? xs[j].y : kNegInf;
                            }
                        }
                        float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                        for (int j = 0; j < kKT / 2; ++j) mx[j & 3] = max3(mx[j & 3], xs[j].x, xs[j].y);
                        top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                    }
                    if (k == k0) {
                        m = top;
                    } else {
                        const bool grown = top - m > 8.0f;
                        if (__any_sync(0xFFFFFFFFu, grown)) {
                            const float f = grown ? ex2(m - top) : 1.0f;
                            if (grown) m = top;
                            l *= f;
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[32];
                                tmem_load32(to + uint32_t(c), o);
                                tmem_wait_ld();
                                tmem_landed32(o);
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_store32(to + uint32_t(c), o);
                            }
                            tmem_wait_st();
                        }
                    }
                    const float mu = m == kNegInf ? 0.0f : m;
                    const float2 sc2 = make_float2(sc, sc), mu2 = make_float2(-mu, -mu);
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    if (Q8) {
                        by_columns(ts, [&](int c, float2 (&x)[32]) {
                            uint32_t p[32];
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const uint4 z = lds128(tv + uint32_t(256 * c + 16 * j));
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    float2 e = __ffma2_rn(x[2 * j + h], sc2, mu2);
                                    e.x = ex2(e.x), e.y = ex2(e.y);
                                    sum[h] = __fadd2_rn(sum[h], e);
                                    e = __fmul2_rn(e, make_float2(__uint_as_float(h ? z.z : z.x), __uint_as_float(h ? z.w : z.y)));
                                    p[2 * j + h] = pack_f16(e.x, e.y);
                                }
                            }
                            tmem_store32(ts + 32u * uint32_t(c), p);  // (columns that have been read)
                        });
                    } else {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t p[32];
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                float2 e = __ffma2_rn(xs[32 * c + j], sc2, mu2);
                                e.x = ex2(e.x), e.y = ex2(e.y);
                                sum[j & 1] = __fadd2_rn(sum[j & 1], e);
                                p[j] = pack_bf16(e.x, e.y);
                            }
                            tmem_store32(ts + 32u * uint32_t(c), p);
                        }
                    }
                    sum[0] = __fadd2_rn(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                    tmem_wait_st();
                }
                if (odd) {
                    if (warp_valid) {
                        if (Q8) clear_weights(scales + (2 * i + 1) % C::kScaleRing * C::kScales, from, until, pos - key0, ts);
                        add_odd<D, Q8>(vb, from, until, pos - key0, ts, to);
                    }
                    bar_any(TWO ? 1 : 2 + slot, TWO ? 256 : 128, false);
                    clear_odd<D, Q8>(vb, from, until, TWO ? int(threadIdx.x) : row, TWO ? 256 : 128);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    bar_any(TWO ? 1 : 2 + slot, TWO ? 256 : 128, false);
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[slot]);
            }

            // ---- the segment's result
            att_wait(&o_done[slot], n_seg++ & 1u, &ctl, a.err);
            tmem_fence_after();
            if (warp_valid) {
                if (valid) ln.part_ml[at] = make_float2(m, l);
                // [channel][row]: a warp's rows are neighbours
                float *dst = ln.part_o + entry * size_t(ln.rt) * D + in_unit;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_load32(to + uint32_t(c), o);
                    tmem_wait_ld();
                    tmem_landed32(o);
                    if (valid)
#pragma unroll
                        for (int j = 0; j < 32; ++j) dst[size_t(c + j) * (TWO ? 256 : 128)] = __uint_as_float(o[j]);
                }
            }
        }
    } else if (Q8 && warp >= kConvWarp) {
        // ---------------------------------------------------- converters
        regs_down<C::kRegsOther>();
        // Units of 128 rows: two warps for the keys, two for the values, so
        // that the next keys do not wait until a values' stage is free.
        constexpr int W = TWO ? 4 : 2;                    // warps per half tile
        const int cw = (warp - kConvWarp) % W;
        // a quarter-warp's 8 lanes read the pieces 0-3 of an even key and 4-7
        // of the next (128 channels), then the others: neither the reads nor
        // the writes of the fp16 pieces share a bank
        const int odd = (lane >> 2) & 1, key = 8 * cw + 2 * (lane >> 3) + odd;  // and 8 W, 16 W .. further
        uint32_t src_at[D / 64], dst_at[D / 64][2];
#pragma unroll
        for (int p = 0; p < D / 64; ++p) {
            const int c = (lane & 3) + (D == 128 ? 4 * (p ^ odd) : 0);
            src_at[p] = D == 128 ? uint32_t(key * 128 + ((c ^ (key & 7)) << 4))
                                 : uint32_t(key * 64 + ((c ^ ((key >> 1) & 3)) << 4));
            const uint32_t row = uint32_t((c >> 2) * kKT * 128 + key * 128);
            const int w = 2 * (c & 3);
            dst_at[p][0] = row + uint32_t((w ^ (key & 7)) << 4);
            dst_at[p][1] = row + uint32_t(((w + 1) ^ (key & 7)) << 4);
        }
        AttSeg seg = sh.first[0];
        int left = seg.left, key0 = seg.key;  // of the segment; the tile's first key
#pragma unroll 1
        for (int h = TWO ? 0 : (warp - kConvWarp) / W; h < 2 * (t1 - t0); h += TWO ? 1 : 2) {  // 2 i + (1 for values)
            if (TWO ? h && !(h & 1) : h > 1) {
                key0 += kKT;
                if (--left == 0) {
                    att_next(a, plan, sh, seg);
                    left = seg.left, key0 = seg.key;
                }
            }
            const int si = h % SI, so = stage(h >> 1, h & 1), turn = used(h >> 1, h & 1), n_keys = seg.key_end - key0;  // keys of the tile (or more)
            const uint32_t src = ring + uint32_t(si) * uint32_t(C::kIn), ss = src + uint32_t(C::kInScale);
            const uint32_t dst = ops + uint32_t(so) * uint32_t(C::kHalf);
            float *sc = scales + (h % C::kScaleRing) * C::kScales;
            const auto put_scales = [&] {
#pragma unroll
                for (int q = 0; q < 4 / W; ++q) {
                    const int k = 32 * (cw + W * q) + lane;
                    sc[k] = k < n_keys ? __uint_as_float(lds32(ss + uint32_t(k) * 4u)) : 0.0f;
                }
            };
            att_wait(&in_full[si], uint32_t(h / SI) & 1u, &ctl, a.err);
            if (h & 1) {  // the softmax takes the values' scales before their product is near
                put_scales();
                if (cw == 0) {  // and their bound
                    uint32_t top = 0u;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float x = __uint_as_float(lds32(ss + uint32_t(32 * q + lane) * 4u));
                        if (x <= 3.0e38f && 32 * q + lane < n_keys) top = max(top, __float_as_uint(x));
                    }
                    top = __reduce_max_sync(0xFFFFFFFFu, top);
                    if (lane == 0) sc[kKT] = exp_above(__uint_as_float(top)) - 7.0f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&vs_full[(h >> 1) % (C::kScaleRing / 2)]);
            }
            if (turn > 0) att_wait(&op_empty[so], uint32_t(turn - 1) & 1u, &ctl, a.err);
            if (!(h & 1)) put_scales();
            // 16-byte pieces of e4m3 rows (16 channels), each to two pieces of
            // the fp16 row; a batch's reads first.  (key & 7) and so the
            // swizzles are the same for every q.
#pragma unroll
            for (int q0 = 0; q0 < 16 / W; q0 += 4) {
                uint4 x[4 * (D / 64)];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int p = 0; p < D / 64; ++p)
                        x[q * (D / 64) + p] = lds128(src + src_at[p] + uint32_t(8 * W * (q0 + q) * D));
                if (n_keys < kKT)  // rows past the end may hold anything
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (key + 8 * W * (q0 + q) >= n_keys)
#pragma unroll
                            for (int p = 0; p < D / 64; ++p) x[q * (D / 64) + p] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int p = 0; p < D / 64; ++p) {
                        const uint4 &y = x[q * (D / 64) + p];
                        const uint32_t to = dst + uint32_t(8 * W * (q0 + q) * 128);
                        sts128(to + dst_at[p][0], e4m3x2_lo_to_f16x2(y.x), e4m3x2_hi_to_f16x2(y.x),
                               e4m3x2_lo_to_f16x2(y.y), e4m3x2_hi_to_f16x2(y.y));
                        sts128(to + dst_at[p][1], e4m3x2_lo_to_f16x2(y.z), e4m3x2_hi_to_f16x2(y.z),
                               e4m3x2_lo_to_f16x2(y.w), e4m3x2_hi_to_f16x2(y.w));
                    }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&op_full[C::kOwn && (h & 3) == 2 ? 3 : so]);
                mbar_arrive(&in_empty[si]);
            }
        }
    } else {
        regs_down<C::kRegsOther>();
        if (warp == kProdWarp || warp == kProdWarp + 3) {
            // -------------------------------------------------------- copies
            // one warp for the keys, one for the values
            const int kv = warp == kProdWarp ? 0 : 1, br = min(a.page, 64);
            int issued = 0;
            att_producer<kKT>(
                a, plan, sh, sh.first[0], br,
                [&](int i) {
                    const int h = 2 * i + kv, s = h % SI;
                    const bool go =
                        h < SI || (att_wait(&in_empty[s], uint32_t(h / SI - 1) & 1u, &ctl, a.err) && !aborted(&ctl));
                    issued += go;
                    return __all_sync(0xFFFFFFFFu, go) != 0;
                },
                [&](int i, int chunks) {
                    mbar_expect_tx(&in_full[(2 * i + kv) % SI], uint32_t(chunks * br) * uint32_t(Q8 ? D + 4 : 2 * D));
                },
                [&](int i, int chunk, int row) {
                    const int s = (2 * i + kv) % SI;
                    const uint32_t st = ring + uint32_t(s) * uint32_t(C::kIn), at = uint32_t(chunk * br);
                    const CUtensorMap *map = kv ? &a.mv : &a.mk;
                    if (Q8) {
                        tma_box(st + at * uint32_t(D), map, 0, row, &in_full[s]);
                        bulk_bytes(st + uint32_t(C::kInScale) + at * 4u, (kv ? a.vs : a.ks) + row, uint32_t(br) * 4u,
                                   &in_full[s]);
                    } else {
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_box(st + uint32_t(x * kKT * 128) + at * 128u, map, 64 * x, row, &in_full[s]);
                    }
                });
            // after a timeout: let the copies in flight land before the CTA ends
            if (lane == 0 && aborted(&ctl))
                for (int j = issued - 1; j >= 0 && j >= issued - SI; --j) {
                    const int h = 2 * j + kv;
                    mbar_drain(&in_full[h % SI], uint32_t(h / SI) & 1u, kAttDrainNs);
                }
        } else if (warp == kIssueWarp || warp == kIssueWarp + 1) {
            // -------------------------------------------------- products
            // A thread per slot.  A burst is P V of a tile and Q K^T of the
            // slot's next.  Units of 256 rows: the two threads take turns by a
            // token, so that the tensor cores finish one slot's scores while
            // the other's warps work on theirs (bursts that interleave end at
            // the same time, and both slots wait at the same time: 110 us
            // without it against 98, 128 requests under a prefix), and each
            // thread's waits -- some 250 cycles even on a barrier that is
            // complete, while products are in flight -- pass under the other's
            // burst.  Units of 128 rows: the slots' tiles alternate anyway
            // (8 x 16 tokens on e4m3: 54.6 us with it, 53.1 without).
            const int slot = warp - kIssueWarp;
            if (lane == 0) {
                const uint32_t iqk = umma_idesc(Q8, kKT, false), ipv = umma_idesc(Q8, D, true);
                const uint32_t ts = tmem + uint32_t(slot) * kSlotCols;
                const uint64_t dq = umma_desc_k(base + uint32_t((TWO ? slot : 0) * (128 * D * 2)));
                uint32_t n_seg = 0, n_p = 0;
                const auto scores = [&](int i, bool pass) {
                    const int s = stage(i, 0);
                    const uint64_t d = umma_desc_k(ops + uint32_t(s) * uint32_t(C::kHalf));
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const uint32_t in_half = 32u * uint32_t(ks & 3);  // 16 channels inside the swizzle atom
                        umma_smem(ts, dq + uint64_t(((ks >> 2) * 128 * 128 + in_half) >> 4),
                                  d + uint64_t(((ks >> 2) * kKT * 128 + in_half) >> 4), iqk, ks ? 1u : 0u);
                        // (the other thread takes its time to see it)
                        if (TWO && ks == KS / 2 - 1 && pass) mbar_arrive(&token[slot ^ 1]);
                    }
                    umma_arrive(&s_full[slot]);
                    umma_arrive(&op_empty[s]);
                };
                AttSeg seg = sh.first[0];
#pragma unroll 1
                for (int t = t0, n; t < t1; t += n) {
                    if (t > t0) att_next(a, plan, sh, seg);
                    const int i0 = t - t0, k0 = first_tile(i0, slot);
                    n = min(seg.left, t1 - t);
                    if (k0 >= n) continue;
                    // (zeros were written to the output, see the softmax warps)
                    const bool zeroed = seg.key + (k0 + 1) * kKT - 1 > att_seen_by_all(a, seg);
                    att_wait(&q_full[slot], n_seg++ & 1u, &ctl, a.err);
                    wait_operand(i0 + k0, 0);
                    tmem_fence_after();
                    scores(i0 + k0, false);
#pragma unroll 1
                    for (int k = k0; k < n; k += kStep) {
                        const int i = i0 + k, s = stage(i, 1);
                        const bool more = k + kStep < n;
                        wait_operand(i, 1);
                        // e4m3: the next keys may be converted only after the
                        // values' stage of a tile before was released
                        if (!Q8 && more) wait_operand(i + kStep, 0);
                        att_wait(&p_full[slot], n_p++ & 1u, &ctl, a.err);
                        if (TWO && (i > 0 || slot))  // burst 2 i + slot
                            att_wait(&token[slot], uint32_t((2 * i + slot - 1) / 2) & 1u, &ctl, a.err);
                        tmem_fence_after();
                        const uint64_t d = umma_desc_mn(ops + uint32_t(s) * uint32_t(C::kHalf), kKT * 128);
#pragma unroll
                        for (int ks = 0; ks < kKT / 16; ++ks) {
                            umma_tmem_a(ts + kOCol, ts + 8u * uint32_t(ks), d + uint64_t((ks * 2048) >> 4), ipv,
                                        (k > k0 || ks || zeroed) ? 1u : 0u);
                            if (TWO && ks == kKT / 32 - 1 && !more) mbar_arrive(&token[slot ^ 1]);
                        }
                        umma_arrive(&op_empty[s]);
                        if (more) {
                            if (Q8) {
                                wait_operand(i + kStep, 0);
                                tmem_fence_after();
                            }
                            scores(i + kStep, true);
                        } else {
                            umma_arrive(&o_done[slot]);
                        }
                    }
                }
                // every product issued has completed before the tensor memory is freed
                umma_arrive(&fin[slot]);
                mbar_drain(&fin[slot], 0u, ctl.limit_ns);
            }
            __syncwarp();
        }
    }
    tmem_fence_before();
    __syncthreads();
    att_end(a);
    if (warp == kIssueWarp) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    }
}

// The dynamic shared-memory limit is raised once per device and variant.
template <int D, bool Q8, bool TWO>
int run(const AttendArgs &a, void *stream) {
    using C = TC<D, Q8, TWO>;
    static std::atomic<uint64_t> ready[4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return W12_ERR_CUDA;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(ready[dev >> 6].load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(attend_tc_kernel<D, Q8, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(C::kSmem)) != cudaSuccess)
            return W12_ERR_CUDA;
        ready[dev >> 6].fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_step(attend_tc_kernel<D, Q8, TWO>, a.line[a.self].grid, C::kThreads, C::kSmem, 1, stream, a);
}

}  // namespace

int launch_attend_tc(const AttendArgs &a, int dim, int kv, void *stream) {
    const bool q8 = kv == W12_KV_E4M3, two = a.line[a.self].rt == 256;
    if (dim == 128)
        return q8 ? (two ? run<128, true, true>(a, stream) : run<128, true, false>(a, stream))
                  : (two ? run<128, false, true>(a, stream) : run<128, false, false>(a, stream));
    return q8 ? (two ? run<64, true, true>(a, stream) : run<64, true, false>(a, stream))
              : (two ? run<64, false, true>(a, stream) : run<64, false, false>(a, stream));
}

}  // namespace w12
