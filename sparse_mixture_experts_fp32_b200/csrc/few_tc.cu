// The layer for a few tokens on tensor cores: bfloat16 and 8-bit experts
// (few.cu describes the call and how blocks share the work).
//
// Both products are D[128 weight rows][columns] = W_tile . B^T: the weights are
// the MMA's 128-row operand, streamed once from memory by TMA, and the columns
// are the tokens of one expert (up to 32), so that an SM's tensor work per
// 16 KB of weights is four MMAs whose cost is reading those 16 KB from shared
// memory: 128 of the about 700 cycles that memory takes to deliver them.  That
// leaves room to spend columns on precision:
//  - bfloat16 experts: a column per token for x; the float32 hidden value h is
//    cut into three bfloat16 terms (exact), a column each;
//  - 8-bit experts run as kind::f8f6f4, weights as e4m3: x in bfloat16 is cut into
//    three e5m2 terms (3 bits each, scaled by 8 more), h into five e4m3 ones (4
//    bits each, scaled by 16 more): each term rounds what the ones before it left.
//    A power of two per token brings its largest value into [2^14, 2^15) or
//    [128, 256).  x takes the wider type, because its 8 bits need three terms of
//    either type once a channel is 2^13 times another, and e5m2's exponents then
//    hold every channel down to 2^-29 of the largest exactly (three e4m3 terms:
//    2^-17).  The epilogue adds the columns of a token with their scales.  (x given
//    in 8 bits is one column as it is.)
// The tensor core truncates each addition to its float32 accumulator: over a
// long row of weights that biases sums by up to 1e-5 (measured: K = 4096, 256
// MMAs in a chain: 4e-6; 16 in a chain: 2.4e-7).  So an accumulator takes four
// ring stages (16 MMAs), and the epilogue warps add accumulators in float32
// registers, rounding to nearest, while the next ones fill.
//
//   warp 0        claims items, loads weight tiles (TMA, 128-byte swizzle) into
//                 a ring of 16 KB stages
//   warp 1        issues the MMAs
//   warps 2-5     epilogue: 32 weight rows each
//   warps 6-11    build the column operands, a stage each: gather x rows,
//                 or add the partial sums of h, apply ReLU and cut into terms
// The ring runs on across items and from the first product into the second:
// weights of the second product are on their way while the first is finished.
// An item is a tile of 128 weight rows of one expert, cut along its length into
// equal parts when there are few tiles (few_splits).
//
// Measured on B200s (whole call in a graph; copy bandwidth 6549 GB/s): 32 tokens
// top-2, 128 bfloat16 experts of 1024 x 4096 152 us (85 % of it), 8 tokens, 64
// 8-bit experts of 4096 x 10240 122 us (79 %): bound by the weights' stream.  One
// token 15.5-16.2 us, 48 tokens top-2 on 8 8-bit experts of 768 x 2048 35.8 us:
// bound by latency (decisions, first weights, the hand-over of h, y from its
// parts), the last by the block that forms y last.
#include <cuda.h>

#include <atomic>

#include "few.cuh"

namespace switchmoe {
namespace {

constexpr int kGroup = 32;        // tokens of a group
constexpr int kStageA = 128 * 128;  // bytes: 128 weight rows x 128 bytes
constexpr int kMaxStages = 12;
constexpr int kRing = 215 * 1024;  // of the 227 KB a block may have: the plan and the barriers take 8 KB
constexpr int kMaxBufs = 8;
constexpr int kChain = 4;         // stages per accumulator
constexpr int kBuilders = 6;      // 4: 3 % slower (32 tokens), 8: 4 % slower (they leave 128 registers a thread)
constexpr int kFull = 60;         // arrivals of a built stage: 60 / w from each of its w <= 6 warps
constexpr int kTcThreads = 32 * (6 + kBuilders);
constexpr int kQueue = 4;
constexpr int kConsumers = 1 + 4 + kBuilders;  // warps that read the item queue

template <bool E4M3, bool X8>
struct Terms {
    static constexpr int first = E4M3 ? (X8 ? 1 : 3) : 1;
    static constexpr int second = E4M3 ? 5 : 3;
};

struct TcShared {
    FewPlan plan;
    uint64_t full_a[kMaxStages], full_b[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[kMaxBufs], acc_empty[kMaxBufs];
    uint64_t q_full[kQueue], q_empty[kQueue];
    uint64_t drain, meet;
    uint32_t tmem;
    int queue[kQueue];
    int ready[kFewMaxA];  // groups whose first product is complete
};

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor for kind::f8f6f4 with e4m3 A, e4m3 or e5m2 B and an fp32 accumulator.
__device__ __forceinline__ uint32_t idesc_e4m3_f32(int M, int N, bool b_e5m2) {
    return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// Parts that the length of a product is cut into: the least of (waves of
// items) x (stages of an item + 1 for its epilogue and hand-over), in half
// stages.  Lane l of the warp weighs 2^l parts.
// Returned as a power of two's exponent.
__device__ __forceinline__ int few_splits(int tiles, int stages, int max_splits, float blocks, int lane) {
    const int log = lane & 7, s = 1 << log;
    const uint32_t waves = (uint32_t)__fdividef((float)(tiles * s) + blocks - 1.f, blocks);
    const uint32_t cost = s <= max_splits && s <= stages ? waves * (2 * ((stages + s - 1) >> log) + 1) : 0xffffffu;
    return (int)(__reduce_min_sync(0xffffffffu, min(cost, 0xffffffu) << 3 | log) & 7);
}

// Work of the call, the same in every block.
struct Work {
    int groups, tiles_h, tiles_o, len_h, len_o, log_h, log_o, splits_h, splits_o, items_h, items;
};
struct Item {
    bool second;
    int g, tile, split, k0, k1;  // ring stages [k0, k1) of the row
};
__device__ __forceinline__ Item locate(const Work &w, int item) {
    Item it;
    it.second = item >= w.items_h;
    if (!it.second) {
        it.split = item & (w.splits_h - 1);
        const int q = item >> w.log_h;
        it.g = q / w.tiles_h;
        it.tile = q - it.g * w.tiles_h;
        it.k0 = it.split * w.len_h >> w.log_h;
        it.k1 = (it.split + 1) * w.len_h >> w.log_h;
    } else {  // all groups' parts of a tile of output rows follow one another
        const int r = item - w.items_h, q = r / w.groups;
        it.g = r - q * w.groups;
        it.split = q & (w.splits_o - 1);
        it.tile = q >> w.log_o;
        it.k0 = it.split * w.len_o >> w.log_o;
        it.k1 = (it.split + 1) * w.len_o >> w.log_o;
    }
    return it;
}

// A flag in shared memory that one thread of the block sets once (release) and others read (acquire).
__device__ __forceinline__ bool ready_cta(const int *flag) {
    int v;
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(smem_u32(flag)) : "memory");
    return v != 0;
}
__device__ __forceinline__ void set_ready_cta(int *flag) {
    asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(smem_u32(flag)), "r"(1) : "memory");
}
__device__ __forceinline__ bool wait_ready_cta(const int *flag, DeviceStatus *st, int32_t where) {
    if (ready_cta(flag)) return true;
    const uint64_t start = global_ns();
    while (!ready_cta(flag)) {
        __nanosleep(20);
        if (global_ns() - start > kWaitLimitNs) {
            report_status(st, SWITCH_ERR_DEVICE_TIMEOUT, where);
            return false;
        }
    }
    return true;
}

// A wait of a whole warp: all its lanes go on or all give up (a limit that ran out for some of them alone would leave
// the others at a shuffle that those never reach).
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, DeviceStatus *st, int32_t where) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, st, where));
}

// Next item from the queue, for one warp; -1: no more, -2: the wait gave up.
__device__ __forceinline__ int next_item(TcShared &s, uint32_t &n, int lane, DeviceStatus *status) {
    const int q = n % kQueue;
    const uint32_t parity = (n / kQueue) & 1u;
    ++n;
    if (!warp_wait(&s.q_full[q], parity, status, 81)) return -2;
    const int item = s.queue[q];
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.q_empty[q]);
    return item;
}

// Power of two that brings a value with these bits into [2^top, 2^(top + 1)) (0
// stays, tiny ones as far as 2^126), as its exponent; 1000: not finite.
constexpr int kTopX = 14, kTopH = 7;
__device__ __forceinline__ int scale_exponent(uint32_t bits, int top) {
    const int e = (int)(bits >> 23) - 127;
    if (bits == 0) return 0;
    return e == 128 ? 1000 : min(126, top - e);
}
__device__ __forceinline__ float pow2(int k) { return __int_as_float((127 + min(127, k)) << 23); }  // k >= -126
__device__ __forceinline__ float unscale(int k) { return k == 1000 ? __int_as_float(0x7fc00000) : pow2(-k); }

// 16 bfloat16 values below 2^15 -> three rows of 16 e5m2 bytes, term i holding
// what the terms before it left, times 8^i.  They are cut in float16, two values
// at a time, which holds every difference exactly: all of the 8 bits of a value
// down to 2^-15; a smaller one is off by half of the third term's smallest step,
// 2^-23, and half of float16's, 2^-25: less than 2^-36 of a row's largest.
__device__ __forceinline__ void store_e5m2_terms(uint8_t *tile, int row0, int chunk, const float (&v)[16]) {
    uint32_t w[3][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        __half2 left = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
#pragma unroll
        for (int t = 0; t < 3; ++t) {
            const __nv_fp8x2_storage_t q = __nv_cvt_halfraw2_to_fp8x2((__half2_raw)left, __NV_SATFINITE, __NV_E5M2);
            if (i & 1) w[t][i >> 1] |= (uint32_t)q << 16;
            else w[t][i >> 1] = q;
            if (t < 2)
                left = __hmul2(__hsub2(left, __half2(__nv_cvt_fp8x2_to_halfraw2(q, __NV_E5M2))), __float2half2_rn(8.f));
        }
    }
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        const int row = row0 + t;
        *reinterpret_cast<uint4 *>(tile + row * 128 + ((chunk ^ (row & 7)) << 4)) =
            make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
    }
}

// 16 values of at most 256 -> five rows of 16 e4m3 bytes, term i holding what
// the terms before it left, times 16^i.  The terms are cut in float16, two
// values at a time: its 11 bits are what three terms hold, down to values of 2^-7
// (below, the third term is at the end of e4m3's range and leaves some); what it
// leaves of v and what they leave of it, times 16^3, make the fourth and fifth.
// So a value is off by 2^-19 of itself, or where that is more by half of the
// fifth term's smallest step, 2^-26, and half of float16's where the fourth
// begins, 2^-29: less than 2^-32 of a row's largest.
__device__ __forceinline__ void store_e4m3_terms(uint8_t *tile, int row0, int chunk, const float (&v)[16]) {
    constexpr int TERMS = 5;
    uint32_t w[TERMS][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        __half2 left = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        const float2 top = __half22float2(left);
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
            if (t == 3)
                left = __hadd2(left, __floats2half2_rn((v[2 * i] - top.x) * 4096.f, (v[2 * i + 1] - top.y) * 4096.f));
            const __nv_fp8x2_storage_t q = __nv_cvt_halfraw2_to_fp8x2((__half2_raw)left, __NV_SATFINITE, __NV_E4M3);
            if (i & 1) w[t][i >> 1] |= (uint32_t)q << 16;
            else w[t][i >> 1] = q;
            if (t + 1 < TERMS)
                left = __hmul2(__hsub2(left, __half2(__nv_cvt_fp8x2_to_halfraw2(q, __NV_E4M3))), __float2half2_rn(16.f));
        }
    }
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
        const int row = row0 + t;
        *reinterpret_cast<uint4 *>(tile + row * 128 + ((chunk ^ (row & 7)) << 4)) =
            make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
    }
}

__device__ __forceinline__ void add4(float *v, const float *p) {
    const float4 a = __ldcg(reinterpret_cast<const float4 *>(p));
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
}

// The column operand of stage `kc` of a first product, x rows: part `part` of
// `team`.
template <bool E4M3, bool X8>
__device__ __forceinline__ void build_x(const FewArgs &p, const FewPlan &s, uint8_t *tile, int a0, int m, int kc,
                                        int my_exp, int lane, int part, int team) {
    const int tasks = m * 8;
    if constexpr (!E4M3 || X8) {  // 16 bytes per task as they are
        const uint8_t *x = static_cast<const uint8_t *>(p.x);
        const int64_t row_bytes = (int64_t)p.d * (E4M3 ? 1 : 2);
        for (int i0 = lane + part * 128; i0 < tasks; i0 += team * 128) {
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u, tok = i >> 3;
                const int64_t at = (int64_t)kc * 128 + (i & 7) * 16;
                v[u] = make_uint4(0, 0, 0, 0);
                if (i < tasks && at < row_bytes)
                    v[u] = __ldg(reinterpret_cast<const uint4 *>(x + (int64_t)s.token[a0 + tok] * row_bytes + at));
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u, row = i >> 3;
                if (i < tasks) *reinterpret_cast<uint4 *>(tile + row * 128 + (((i & 7) ^ (row & 7)) << 4)) = v[u];
            }
        }
    } else {
        const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(p.x);
        for (int i0 = part * 32; i0 < tasks; i0 += team * 32) {  // whole warps: the exponents are exchanged
            const int i = i0 + lane, tok = i >> 3, at = kc * 128 + (i & 7) * 16;
            const float up = pow2(__shfl_sync(0xffffffffu, my_exp, tok & 31));
            if (i >= tasks) continue;
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.f;
            if (at < p.d) {
                const uint4 *src = reinterpret_cast<const uint4 *>(x + (int64_t)s.token[a0 + tok] * p.d + at);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 a = __ldg(src + h);
                    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[8 * h + 2 * j] = __uint_as_float(w[j] << 16) * up;
                        v[8 * h + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * up;
                    }
                }
            }
            store_e5m2_terms(tile, tok * 3, i & 7, v);
        }
    }
}

// V values of a pair's hidden row from `src` on: its parts summed in order.
template <int V>
__device__ __forceinline__ void load_h(const float *src, int64_t step, int splits, float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
        const float4 a = __ldcg(reinterpret_cast<const float4 *>(src) + j);
        v[4 * j] = a.x, v[4 * j + 1] = a.y, v[4 * j + 2] = a.z, v[4 * j + 3] = a.w;
    }
#pragma unroll 4
    for (int q = 1; q < splits; ++q)
#pragma unroll
        for (int j = 0; j < V / 4; ++j) add4(v + 4 * j, src + q * step + 4 * j);
}

// The column operand of stage `kc` of a second product, ReLU of h in terms:
// part `part` of `team`.
template <bool E4M3>
__device__ __forceinline__ void build_h(const FewArgs &p, uint8_t *tile, int A, int splits, int a0, int m, int kc,
                                        int my_exp, int lane, int part, int team) {
    constexpr int V = E4M3 ? 16 : 8;  // values per 16-byte chunk
    const int tasks = m * 8, at = (kc * 8 + (lane & 7)) * V;
    const bool in = at < p.F;
    const float *h = p.h + (int64_t)a0 * p.F + at;
    const int64_t step = (int64_t)A * p.F;
    float next[V];
    const int stride = team * 32;
    int i = part * 32 + lane;
    if (i < tasks && in) load_h<V>(h + (int64_t)(i >> 3) * p.F, step, splits, next);
    for (int i0 = part * 32; i0 < tasks; i0 += stride, i += stride) {
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = next[j];
        // the following task's values are on their way while this one's are cut
        if (i + stride < tasks && in) load_h<V>(h + (int64_t)((i + stride) >> 3) * p.F, step, splits, next);
        const int tok = i >> 3;
        const float up = E4M3 ? pow2(__shfl_sync(0xffffffffu, my_exp, tok & 31)) : 1.f;
        if (i >= tasks) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = !in || v[j] < 0.f ? 0.f : v[j] * up;  // NaN stays NaN
        if constexpr (E4M3) {
            store_e4m3_terms(tile, tok * 5, lane & 7, v);
        } else {
            uint16_t t[3][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint16_t c[3];
                split_bf16x3(v[j], c);
                t[0][j] = c[0], t[1][j] = c[1], t[2][j] = c[2];
            }
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                const int row = tok * 3 + c;
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = (uint32_t)t[c][2 * j] | ((uint32_t)t[c][2 * j + 1] << 16);
                *reinterpret_cast<uint4 *>(tile + row * 128 + (((lane & 7) ^ (row & 7)) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// v[j] += the accumulator's value for token j (its terms joined, each STEP times the one before it), m tokens.
template <int TERMS, int STEP>
__device__ __forceinline__ void add_accumulator(uint32_t taddr, int m, float (&v)[kGroup]) {
#pragma unroll
    for (int b = 0; b < kGroup / 8; ++b) {
        if (b * 8 >= m) break;
        uint32_t r[TERMS][8];
#pragma unroll
        for (int t = 0; t < TERMS; ++t) tmem_ld_32x32b_x8(taddr + (uint32_t)((b * TERMS + t) * 8), r[t]);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a = 0.f;  // from the smallest term up
#pragma unroll
            for (int t = TERMS - 1; t >= 0; --t) {
                const int col = j * TERMS + t;
                a = a * (1.f / STEP) + __uint_as_float(r[col / 8][col % 8]);
            }
            v[b * 8 + j] += a;
        }
    }
}

// y of one output row for the first B tokens of `mask` (positions from a0 on),
// whose parts are all there; returns the mask without them.  The loads of U
// parts of all choices of all B tokens are in flight together.
template <int B, int U, int K>
__device__ __forceinline__ uint32_t combine_tokens(const FewArgs &p, const FewPlan &s, int splits, int step, int a0,
                                                   uint32_t mask, int row) {
    int t[B], at[B][K];  // (512 rows of 8192 values at most: 32-bit offsets)
    float o[B][K];
    const float *src = p.o + row;
#pragma unroll
    for (int u = 0; u < B; ++u) {
        t[u] = s.token[a0 + __ffs(mask) - 1];  // past the last one: the last one again
        if (u == B - 1 || (mask & (mask - 1))) mask &= mask - 1;
#pragma unroll
        for (int c = 0; c < K; ++c) at[u][c] = max(s.pos[t[u] * K + c], 0) * p.d, o[u][c] = 0.f;
    }
#pragma unroll U
    for (int q = 0; q < splits; ++q)
#pragma unroll
        for (int u = 0; u < B; ++u)
#pragma unroll
            for (int c = 0; c < K; ++c) o[u][c] += __ldcg(src + at[u][c] + q * step);
#pragma unroll
    for (int u = 0; u < B; ++u) {
        float y = 0.f;
#pragma unroll
        for (int c = 0; c < K; ++c)
            if (s.pos[t[u] * K + c] >= 0) y += s.gate[t[u] * K + c] * o[u][c];
        p.y[(int64_t)t[u] * p.d + row] = y;
    }
    return mask;
}

template <int K>
__device__ __forceinline__ void combine_row(const FewArgs &p, const FewPlan &s, int splits, int A, int a0,
                                            uint32_t mask, int row) {
    const int step = A * p.d;
    while (mask) {
        const int n = __popc(mask);
        mask = n == 1 ? combine_tokens<1, 8, K>(p, s, splits, step, a0, mask, row)
               : n <= 4 ? combine_tokens<4, 8 / K, K>(p, s, splits, step, a0, mask, row)
                        : combine_tokens<8, 4 / K, K>(p, s, splits, step, a0, mask, row);
    }
}

// max_splits: parts of h and o that the workspace holds.
template <bool E4M3, bool X8>
__global__ void __launch_bounds__(kTcThreads, 1)
    few_experts_tc_kernel(const __grid_constant__ CUtensorMap tmap_in, const __grid_constant__ CUtensorMap tmap_out,
                          const FewArgs p, int max_splits) {
    extern __shared__ uint8_t raw[];
    __shared__ TcShared s;
    uint8_t *ring_a = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int A = p.T * p.k;
    if (warp == 1) {
        if (lane == 0) {
            for (int i = 0; i < kMaxStages; ++i) {
                mbar_init(&s.full_a[i], 1);
                mbar_init(&s.full_b[i], kFull);
                mbar_init(&s.empty[i], 1);
            }
            for (int i = 0; i < kMaxBufs; ++i) {
                mbar_init(&s.acc_full[i], 1);
                mbar_init(&s.acc_empty[i], 4);
            }
            for (int i = 0; i < kQueue; ++i) {
                mbar_init(&s.q_full[i], 1);
                mbar_init(&s.q_empty[i], kConsumers);
            }
            mbar_init(&s.drain, 1);
            mbar_init(&s.meet, 4);
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc(&s.tmem, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    if (tid < kFewMaxA) s.ready[tid] = 0;
    if (tid == 0) {
        prefetch_tmap(&tmap_in);
        prefetch_tmap(&tmap_out);
    }
    pdl_wait();  // the logits and the zeroed counters
    int claimed = 0;
    if (tid == 0) claimed = atomicAdd(&p.ctr->claim, 1);
    few_plan(p, s.plan, kGroup, kTcThreads);
    Work w;
    w.groups = s.plan.groups;
    w.tiles_h = (p.F + 127) / 128;
    w.tiles_o = (p.d + 127) / 128;
    w.len_h = (p.d * (E4M3 ? 1 : 2) + 127) / 128;
    w.len_o = (p.F * (E4M3 ? 1 : 2) + 127) / 128;
    w.log_h = few_splits(w.groups * w.tiles_h, w.len_h, max_splits, (float)gridDim.x, lane);
    w.log_o = few_splits(w.groups * w.tiles_o, w.len_o, max_splits, (float)gridDim.x, lane);
    w.splits_h = 1 << w.log_h;
    w.splits_o = 1 << w.log_o;
    w.items_h = w.groups * w.tiles_h << w.log_h;
    w.items = w.items_h + (w.groups * w.tiles_o << w.log_o);
    // The ring and the accumulators are laid out for the call's largest group:
    // bytes of a stage's column operand (whole 8-row swizzle atoms), stages, columns and number of accumulators.
    constexpr int kTerms = Terms<E4M3, X8>::second;  // the larger of the two products'
    const int b_bytes = (s.plan.largest * kTerms + 15) / 16 * 16 * 128;
    const int stages = min(kMaxStages, kRing / (kStageA + b_bytes));
    const int acc_cols = ((s.plan.largest + 7) / 8 * 8 * kTerms + 31) / 32 * 32;
    const int bufs = min(512 / acc_cols, kMaxBufs);
    uint8_t *ring_b = ring_a + stages * kStageA;
    tc_fence_after();  // the plan's barriers stand between the allocation and here
    const uint32_t tmem = s.tmem;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, issued = 0, parity_of = 0;
            bool ok = true;
            for (uint32_t n = 0; ok; ++n) {
                const int q = n % kQueue, item = claimed;
                if (!mbar_wait(&s.q_empty[q], ((n / kQueue) & 1u) ^ 1u, p.status, 82)) break;
                s.queue[q] = item < w.items ? item : -1;
                mbar_arrive(&s.q_full[q]);
                if (item >= w.items) break;
                // The next item's claim runs while this one's loads are issued.  Where the second product has an
                // item per block at most, a block takes one: a second, claimed ahead by a block that waits, would
                // come after it while other blocks have none.
                const bool last = item >= w.items_h && w.items - w.items_h <= (int)gridDim.x;
                claimed = last ? w.items : atomicAdd(&p.ctr->claim, 1);
                const Item it = locate(w, item);
                const int e = s.plan.g_expert[it.g];
                for (int kc = it.k0; kc < it.k1; ++kc) {
                    if (!mbar_wait(&s.empty[stage], phase ^ 1u, p.status, 83)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&s.full_a[stage], kStageA);
                    tma_load_3d(ring_a + stage * kStageA, it.second ? &tmap_out : &tmap_in, &s.full_a[stage],
                                kc * (E4M3 ? 128 : 64), it.tile * 128, e);
                    issued |= 1u << stage;
                    parity_of = (parity_of & ~(1u << stage)) | (phase << stage);
                    if (++stage == stages) stage = 0, phase ^= 1u;
                }
            }
            // every load has landed before the block may end
            for (int i = 0; i < stages; ++i)
                if (issued & (1u << i)) mbar_wait(&s.full_a[i], (parity_of >> i) & 1u, p.status, 84);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, acc_phase = 0, n = 0;
            bool ok = true;
            while (ok) {
                const int q = n % kQueue;
                if (!mbar_wait(&s.q_full[q], (n / kQueue) & 1u, p.status, 85)) break;
                const int item = s.queue[q];
                mbar_arrive(&s.q_empty[q]);
                ++n;
                if (item < 0) break;
                const Item it = locate(w, item);
                const int cols = s.plan.g_size[it.g] * (it.second ? Terms<E4M3, X8>::second : Terms<E4M3, X8>::first);
                const int N = (cols + 15) / 16 * 16;
                const uint32_t idesc = E4M3 ? idesc_e4m3_f32(128, N, !X8 && !it.second) : idesc_bf16_f32(128, N);
                for (int kc = it.k0; ok && kc < it.k1;) {
                    if (!mbar_wait(&s.acc_empty[buf], acc_phase ^ 1u, p.status, 86)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(buf * acc_cols);
                    const int end = min(kc + kChain, it.k1);
                    for (uint32_t more = 0; kc < end; ++kc) {
                        if (!mbar_wait(&s.full_a[stage], phase, p.status, 87) ||
                            !mbar_wait(&s.full_b[stage], phase, p.status, 88)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t a_desc = smem_desc_sw128(ring_a + stage * kStageA);
                        const uint64_t b_desc = smem_desc_sw128(ring_b + stage * b_bytes);
#pragma unroll
                        for (int k = 0; k < 4; ++k, more = 1) {  // 32 bytes of every row each
                            if constexpr (E4M3) tc_mma_f8(d, a_desc + 2 * k, b_desc + 2 * k, idesc, more);
                            else tc_mma_bf16(d, a_desc + 2 * k, b_desc + 2 * k, idesc, more);
                        }
                        tc_commit(&s.empty[stage]);
                        if (++stage == stages) stage = 0, phase ^= 1u;
                    }
                    if (!ok) break;
                    tc_commit(&s.acc_full[buf]);
                    if (++buf == bufs) buf = 0, acc_phase ^= 1u;
                }
            }
            tc_commit(&s.drain);
            mbar_wait(&s.drain, 0, p.status, 89);
        }
    } else if (warp < 6) {
        const int quarter = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const bool direct = p.k == 1 && w.splits_o == 1;  // an item's output rows are y's
        int buf = 0;
        uint32_t acc_phase = 0, n = 0;
        bool ok = true, gates = false;
        // While the first weights are on their way; with at most one item of the first product per block
        // between the products, when its last parts are on their way through other blocks.
        const bool late = w.items_h <= (int)gridDim.x;
        while (ok) {
            const int item = late || gates ? next_item(s, n, lane, p.status) : 0;
            if (item == -2) break;
            if (!gates && (!late || item < 0 || item >= w.items_h)) {
                gates = true;
                // (a barrier that gives up: one of the four warps may have left after a wait of its own did)
                uint32_t turn = 0;
                ok = few_gates(p, s.plan, tid - 64, blockIdx.x == 0, [&] {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.meet);
                    const bool met = warp_wait(&s.meet, turn, p.status, 94);
                    turn ^= 1u;
                    return met;
                });
                if (!ok) break;
                for (int t = blockIdx.x; t < p.T; t += gridDim.x)  // tokens that no expert keeps
                    if (s.plan.pos[t * p.k] < 0 && s.plan.pos[t * p.k + p.k - 1] < 0)
                        for (int j = tid - 64; j < p.d; j += 128) p.y[(int64_t)t * p.d + j] = 0.f;
                if (!late) continue;
            }
            if (item < 0) break;
            const Item it = locate(w, item);
            const int e = s.plan.g_expert[it.g], a0 = s.plan.g_first[it.g], m = s.plan.g_size[it.g];
            const int row = it.tile * 128 + quarter * 32 + lane, rows = it.second ? p.d : p.F;
            const bool live = row < rows;
            float v[kGroup];
#pragma unroll
            for (int j = 0; j < kGroup; ++j) v[j] = 0.f;
            float scale = 1.f, own = 1.f;  // of the weight row; of token `lane` of the group
            if constexpr (E4M3) {
                if (live) scale = __ldg((it.second ? p.w_out_scale : p.w_in_scale) + (int64_t)e * rows + row);
                if (!it.second && lane < m) {
                    const int t = s.plan.token[a0 + lane];
                    own = X8 ? __ldg(p.x_scale + t) : unscale(scale_exponent(__ldcg(p.xmax + t), kTopX));
                }
            }
            for (int kc = it.k0; kc < it.k1; kc += kChain) {
                if (!warp_wait(&s.acc_full[buf], acc_phase, p.status, 90)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = lanes + (uint32_t)(buf * acc_cols);
                if (it.second) add_accumulator<Terms<E4M3, X8>::second, E4M3 ? 16 : 1>(at, m, v);
                else add_accumulator<Terms<E4M3, X8>::first, E4M3 ? 8 : 1>(at, m, v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.acc_empty[buf]);
                if (++buf == bufs) buf = 0, acc_phase ^= 1u;
            }
            if (!ok) break;
            if constexpr (E4M3) {
                // an accumulator of the second product exists once every part of h does: so do their maxima
                if (it.second && lane < m) {
                    float top = 0.f;
                    for (int q = 0; q < w.splits_h; ++q) top += __uint_as_float(__ldcg(p.hmax + q * A + a0 + lane));
                    own = unscale(scale_exponent(__float_as_uint(top), kTopH));
                }
            }
            float *out = it.second ? p.o + ((int64_t)it.split * A + a0) * p.d : p.h + ((int64_t)it.split * A + a0) * p.F;
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                if (j >= m) break;
                float u = v[j];
                if constexpr (E4M3) {
                    u = u * __shfl_sync(0xffffffffu, own, j) * scale;
                    if (!it.second) {
                        // Negative values are left out: ReLU removes them, or the sum with other parts is less than
                        // theirs.  (A NaN's bits are above all.)
                        const uint32_t top =
                            __reduce_max_sync(0xffffffffu, live && !(u < 0.f) ? __float_as_uint(u) & 0x7fffffffu : 0u);
                        if (lane == 0) atomicMax(p.hmax + it.split * A + a0 + j, top);
                    }
                }
                if (live) {
                    if (it.second && direct) {
                        const int t = s.plan.token[a0 + j];
                        p.y[(int64_t)t * p.d + row] = s.plan.gate[t] * u;
                    } else {
                        out[(int64_t)j * rows + row] = u;
                    }
                }
            }
            __syncwarp();
            if (!it.second) {
                if (lane == 0) red_release_add_gpu(&p.ctr->done[it.g], 1);
            } else if (!direct) {  // the warp that stores the last part of a token's values forms them
                bool last = false;
                if (lane < m) {
                    const int t = s.plan.token[a0 + lane];
                    const int kept = (s.plan.pos[t * p.k] >= 0) + (p.k == 2 && s.plan.pos[t * p.k + 1] >= 0);
                    last = atom_add_acq_rel_gpu(p.parts + (int64_t)(it.tile * 4 + quarter) * p.T + t, 1) ==
                           kept * w.splits_o - 1;
                }
                const uint32_t mask = __ballot_sync(0xffffffffu, last);
                __syncwarp();  // the other warps' parts, which a lane has acquired, are read by all (a ballot orders no memory)
                if (mask && live) {
                    if (p.k == 1) combine_row<1>(p, s.plan, w.splits_o, A, a0, mask, row);
                    else combine_row<2>(p, s.plan, w.splits_o, A, a0, mask, row);
                }
                __syncwarp();
            }
        }
    } else {
        // Stage i of an item is built by warp i mod `builders`, or by several where the item has fewer stages than
        // there are warps.  A warp may take the parity of an older phase for that of the one it waits for once it is
        // a whole lap of the ring ahead; it is not: the producer hands out an item after it has claimed the ring for
        // all items before, which covers the first `stages` stages of this one, and from there on a warp's own
        // stages lie `builders` <= `stages` apart.
        const int builders = min(kBuilders, stages), me = warp - 6;
        int base = 0;  // ring stage and phase of the item's first stage
        uint32_t base_phase = 0, n = 0;
        bool ok = true;
        while (ok) {
            const int item = next_item(s, n, lane, p.status);
            if (item < 0) break;
            const Item it = locate(w, item);
            const int a0 = s.plan.g_first[it.g], m = s.plan.g_size[it.g], len = it.k1 - it.k0;
            // One warp of the block asks memory whether the group's first product is complete, the others that one; in a
            // warp one lane does, for all (lanes that read the flag at different times must not part ways).
            if (it.second) {
                int fine = 1;
                if (lane == 0 && !ready_cta(&s.ready[it.g])) {
                    if (me == 0) {
                        fine = wait_counter_geq(&p.ctr->done[it.g], 4 * w.tiles_h << w.log_h, p.status, 91);
                        if (fine) set_ready_cta(&s.ready[it.g]);
                    } else {
                        fine = wait_ready_cta(&s.ready[it.g], p.status, 93);
                    }
                }
                ok = __shfl_sync(0xffffffffu, fine, 0) != 0;
                if (!ok) break;
                __syncwarp();  // what lane 0 has acquired, the others may read
            }
            const int team = len >= builders ? 1 : builders / len;
            int first = me / team;
            const int part = me - first * team;
            if (me >= builders) first = len;
            if (first < len) {
                int my_exp = 0;  // 8-bit experts: exponent of token `lane`'s scale
                if constexpr (E4M3) {
                    if (lane < m) {
                        if (it.second) {
                            float top = 0.f;
                            for (int q = 0; q < w.splits_h; ++q)
                                top += __uint_as_float(__ldcg(p.hmax + q * A + a0 + lane));
                            my_exp = scale_exponent(__float_as_uint(top), kTopH);
                        } else if (!X8) {
                            my_exp = scale_exponent(__ldcg(p.xmax + s.plan.token[a0 + lane]), kTopX);
                        }
                    }
                }
                int stage = base + first;
                uint32_t phase = base_phase;
                for (int i = first; i < len; i += builders, stage += builders) {
                    while (stage >= stages) stage -= stages, phase ^= 1u;
                    if (!warp_wait(&s.empty[stage], phase ^ 1u, p.status, 92)) {
                        ok = false;
                        break;
                    }
                    uint8_t *tile = ring_b + stage * b_bytes;
                    if (it.second) build_h<E4M3>(p, tile, A, w.splits_h, a0, m, it.k0 + i, my_exp, lane, part, team);
                    else build_x<E4M3, X8>(p, s.plan, tile, a0, m, it.k0 + i, my_exp, lane, part, team);
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_n(&s.full_b[stage], kFull / team);
                }
            }
            base += len;
            while (base >= stages) base -= stages, base_phase ^= 1u;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// [E][rows][K] weights, box = 128 rows x 128 bytes, 128-byte swizzle; zeros past an expert's rows and K.
bool weight_map(CUtensorMap *map, const void *ptr, int E, int rows, int K, bool e4m3) {
    const EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t size = e4m3 ? 1 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)rows, (cuuint64_t)E};
    const cuuint64_t strides[2] = {(cuuint64_t)K * size, (cuuint64_t)rows * K * size};
    const cuuint32_t box[3] = {e4m3 ? 128u : 64u, 128u, 1u}, unit[3] = {1, 1, 1};
    return fn(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr),
              dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool E4M3, bool X8>
cudaError_t experts_tc(const FewArgs &p, int max_splits, cudaStream_t stream) {
    CUtensorMap in, out;
    if (!weight_map(&in, p.w_in, p.N, p.F, p.d, E4M3) || !weight_map(&out, p.w_out, p.N, p.d, p.F, E4M3))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> raised{0};  // devices whose limit is raised already, a bit each
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
        err = cudaFuncSetAttribute(few_experts_tc_kernel<E4M3, X8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   1024 + kRing);
        if (err != cudaSuccess) return err;
        raised.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_kernel(few_experts_tc_kernel<E4M3, X8>, dim3(device_sm_count()), dim3(kTcThreads), 1024 + kRing,
                         stream, true, in, out, p, max_splits);
}

}  // namespace

cudaError_t launch_few_experts_tc(const FewArgs &p, int w_dtype, int x_dtype, int max_splits, cudaStream_t stream) {
    launch_begin(K_FEW_EXPERTS_TC, stream);
    cudaError_t err;
    if (w_dtype == SWITCH_BF16) err = experts_tc<false, false>(p, max_splits, stream);
    else if (x_dtype == SWITCH_E4M3) err = experts_tc<true, true>(p, max_splits, stream);
    else err = experts_tc<true, false>(p, max_splits, stream);
    launch_end(stream);
    return err;
}

}  // namespace switchmoe
