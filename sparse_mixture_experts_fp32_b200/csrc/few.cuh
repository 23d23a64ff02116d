// The layer for a few tokens: what its kernels share (sizes, workspace,
// the routing decisions every block forms for itself, the claim of work).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace switchmoe {

constexpr int kFewMaxT = SWITCH_FEW_MAX_TOKENS;
constexpr int kFewMaxA = 2 * kFewMaxT;  // (token, choice) pairs
constexpr int kFewMaxN = 256;

// Counters, zeroed by the router kernel of the same call.
struct FewCounters {
    int32_t claim;                 // next item of work
    int32_t pad[3];
    int32_t done[kFewMaxA];        // finished items of a group's first product
    int32_t tile[1024];            // finished items of a tile of output rows
};

struct FewArgs {
    int T, d, F, N, C, k;
    const void *x;
    const float *x_scale, *w_r, *bias;
    const void *w_in, *w_out;
    const float *w_in_scale, *w_out_scale;
    float *y, *gate, *aux;
    int32_t *expert, *slot, *counts;
    // workspace
    DeviceStatus *status;
    FewCounters *ctr;
    uint32_t *xmax;    // [T] bits of max |x| (8-bit experts with bfloat16 x)
    uint32_t *hmax;    // [splits][A] bits of the largest positive partial sum of a pair's hidden row (tensor cores); their
                       // sum over the parts is at least the row's largest value after ReLU
    int32_t *parts;    // [ceil(d / 128) * 4][T] finished parts of 32 values of a token's y (tensor cores)
    float *logits;     // [T][N]
    float *h;          // [splits][A][F] first product (before ReLU where it is split)
    float *o;          // [splits][A][d] second product
};

// The routing decisions, in shared memory.  Pairs (token, choice) that are
// kept get consecutive positions ("a"), by expert and slot; a group is up to
// `group_max` positions of one expert.
struct FewPlan {
    int expert[kFewMaxA];    // [t * k + c]
    float gate[kFewMaxA];    // [t * k + c]
    int slot[kFewMaxA];      // [t * k + c], -1: dropped
    int pos[kFewMaxA];       // [t * k + c] -> position, -1: dropped
    int token[kFewMaxA];     // [position] -> token
    // an entry per pair, first choices (in token order) before second ones
    uint32_t order[kFewMaxA / 4];  // its expert, a byte each
    uint32_t keeps[kFewMaxA / 4];  // 0xff where it is kept
    int lead[kFewMaxA];      // [position] size of the group that begins there, 0: none does
    int lead_expert[kFewMaxA];
    int g_expert[kFewMaxA], g_first[kFewMaxA], g_size[kFewMaxA];
    int cnt[kFewMaxN], first[kFewMaxN];  // pairs and first choices of each expert (the block that writes the outputs)
    double aux[4];
    int groups, largest;     // groups; positions of the largest one
};

// Bits whose unsigned order is the order of floats; NaN is below everything.
__device__ __forceinline__ uint32_t ordered_bits(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 and 0 tie
    return v != v ? 0u : b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ void few_logits(const FewArgs &p, int t, int lane, float (&v)[kFewMaxN / 32]) {
#pragma unroll
    for (int i = 0; i < kFewMaxN / 32; ++i) {
        const int n = 32 * i + lane;
        v[i] = n < p.N ? __ldcg(p.logits + (int64_t)t * p.N + n) : -INFINITY;
    }
}

// Of a warp's keys: the largest, and the lowest index that has it.
__device__ __forceinline__ int few_argmax(uint32_t key, int index) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, key);
    return (int)__reduce_min_sync(0xffffffffu, key == best ? (uint32_t)index : 0xffffu);
}

// Every thread of a block of `threads` (a multiple of 32, at least 256) calls
// this.  T and N are small (64 x 256 logits at most), so that every block
// deciding for itself costs less than another kernel or a grid-wide wait would.
// It stands before the first weight that a block can ask for, so it does only
// what the work list needs: the gates are few_gates', later.
__device__ inline void few_plan(const FewArgs &p, FewPlan &s, int group_max, int threads) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = threads >> 5;
    const int A = p.T * p.k;
    if (tid < kFewMaxA) {
        s.lead[tid] = 0;
        if (tid >= A) reinterpret_cast<uint8_t *>(s.order)[tid] = 0xff;
    }
    float v[kFewMaxN / 32];
    if (warp < p.T) few_logits(p, warp, lane, v);
#pragma unroll 1
    for (int t = warp; t < p.T; t += warps) {
        uint32_t k1 = 0, k2 = 0;  // this lane's two largest keys, the lower index first among equals
        int n1 = 0xffff, n2 = 0xffff;
#pragma unroll
        for (int i = 0; i < kFewMaxN / 32; ++i) {
            if (32 * i >= p.N) break;
            const int n = 32 * i + lane;
            const uint32_t key = n < p.N ? ordered_bits(v[i]) : 0u;
            if (n < p.N && (key > k1 || n1 == 0xffff)) k2 = k1, n2 = n1, k1 = key, n1 = n;
            else if (n < p.N && (key > k2 || n2 == 0xffff)) k2 = key, n2 = n;
        }
        if (t + warps < p.T) few_logits(p, t + warps, lane, v);
        const int first = few_argmax(k1, n1);
        const int second = p.k == 2 ? few_argmax(n1 == first ? k2 : k1, n1 == first ? n2 : n1) : 0;
        if (lane == 0) {
            s.expert[t * p.k] = first;
            reinterpret_cast<uint8_t *>(s.order)[t] = (uint8_t)first;
            if (p.k == 2) {
                s.expert[2 * t + 1] = second;
                reinterpret_cast<uint8_t *>(s.order)[p.T + t] = (uint8_t)second;
            }
        }
    }
    __syncthreads();
    // Entry i: the entries of its expert before it (its rank, its slot where it is kept), of its expert, and of
    // lower experts; four at a time.
    const bool mine = tid < A;
    const int c = tid >= p.T, t = c ? tid - p.T : tid;
    int e = 0, rank = 0, same = 0, lower = 0;
    if (mine) {
        e = s.expert[t * p.k + c];
        const uint32_t four = (uint32_t)e * 0x01010101u;
        // (a byte of a comparison is -1 where it holds; bytes past the last entry are 0xff)
#pragma unroll 4
        for (int w = 0; 4 * w < A; ++w) {
            const uint32_t eq = __vcmpeq4(s.order[w], four);
            const int n = -__dp4a((int)eq, 0x01010101, 0);
            same += n;
            if (4 * w + 4 <= tid) rank += n;
            lower -= __dp4a((int)__vcmpltu4(s.order[w], four), 0x01010101, 0);
        }
        if (tid & 3) rank += __popc(__vcmpeq4(s.order[tid >> 2], four) & ((1u << (8 * (tid & 3))) - 1u)) >> 3;
        if (e == 255) same -= -A & 3;
    }
    const bool keep = mine && rank < p.C;
    if (p.C < p.T) {  // some may be dropped: count the kept ones of lower experts again
        if (mine) reinterpret_cast<uint8_t *>(s.keeps)[tid] = keep ? 0xff : 0;
        __syncthreads();
        if (keep) {
            const uint32_t four = (uint32_t)e * 0x01010101u;
            lower = 0;
            for (int w = 0; 4 * w < A; ++w)
                lower -= __dp4a((int)(__vcmpltu4(s.order[w], four) & s.keeps[w]), 0x01010101, 0);
        }
    }
    if (mine) {
        s.slot[t * p.k + c] = keep ? rank : -1;
        s.pos[t * p.k + c] = keep ? lower + rank : -1;
        if (keep) {
            s.token[lower + rank] = t;
            if (rank % group_max == 0) {
                s.lead[lower + rank] = min(group_max, min(same, p.C) - rank);
                s.lead_expert[lower + rank] = e;
            }
        }
    }
    __syncthreads();
    if (warp == 0) {
        int groups = 0, largest = 0;
#pragma unroll
        for (int q = 0; q < kFewMaxA / 32; ++q) {
            const int a = 32 * q + lane, size = s.lead[a];
            const uint32_t leads = __ballot_sync(0xffffffffu, size > 0);
            if (size > 0) {
                const int g = groups + __popc(leads & ((1u << lane) - 1u));
                s.g_expert[g] = s.lead_expert[a];
                s.g_first[g] = a;
                s.g_size[g] = size;
            }
            groups += __popc(leads);
            largest = max(largest, size);
        }
        largest = __reduce_max_sync(0xffffffffu, largest);
        if (lane == 0) s.groups = groups, s.largest = largest;
    }
    __syncthreads();
}

// The gates, by four warps (`tid` = 0..127) for which meet() is a barrier; with
// `outputs` (one block) the call's routing outputs too.  meet() returns false
// where it gave up, and so does this.
// aux = N / T^2 sum_t sum_n f_n p_tn, f_n the first choices of expert n:
// float64, in a fixed order.
template <typename Meet>
__device__ __forceinline__ bool few_gates(const FewArgs &p, FewPlan &s, int tid, bool outputs, Meet meet) {
    const int warp = tid >> 5, lane = tid & 31;
    double aux = 0.0;
    if (outputs) {
        for (int n = tid; n < p.N; n += 128) s.cnt[n] = s.first[n] = 0;
        if (!meet()) return false;
        for (int i = tid; i < p.T * p.k; i += 128) {
            atomicAdd(&s.cnt[s.expert[i]], 1);
            if (p.k == 1 || (i & 1) == 0) atomicAdd(&s.first[s.expert[i]], 1);
        }
        if (!meet()) return false;
    }
    float v[kFewMaxN / 32], next[kFewMaxN / 32];
    if (warp < p.T) few_logits(p, warp, lane, next);
#pragma unroll 1
    for (int t = warp; t < p.T; t += 4) {
        float top, l = 0.f;  // lane c: the logit of choice c
        const int mine = s.expert[t * p.k + (lane < p.k ? lane : 0)];
#pragma unroll
        for (int i = 0; i < kFewMaxN / 32; ++i) v[i] = next[i];
        if (t + 4 < p.T) few_logits(p, t + 4, lane, next);
#pragma unroll
        for (int i = 0; i < kFewMaxN / 32; ++i) {
            if (32 * i >= p.N) break;
            const float u = __shfl_sync(0xffffffffu, v[i], mine & 31);
            if (mine >> 5 == i) l = u;
        }
        top = __shfl_sync(0xffffffffu, l, 0);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kFewMaxN / 32; ++i) {
            if (32 * i >= p.N) break;
            v[i] = 32 * i + lane < p.N ? expf(v[i] - top) : 0.f;
            sum += v[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane < p.k) s.gate[t * p.k + lane] = expf(l - top) / sum;  // NaN for a token whose logits are not finite
        if (outputs) {
#pragma unroll
            for (int i = 0; i < kFewMaxN / 32; ++i) {
                if (32 * i >= p.N) break;
                const int f = 32 * i + lane < p.N ? s.first[32 * i + lane] : 0;
                if (f) aux += (double)f * (double)(v[i] / sum);
            }
        }
    }
    if (outputs) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) aux += __shfl_xor_sync(0xffffffffu, aux, o);
        if (lane == 0) s.aux[warp] = aux;
    }
    if (!meet()) return false;
    if (outputs) {
        for (int i = tid; i < p.T * p.k; i += 128)
            p.expert[i] = s.expert[i], p.gate[i] = s.gate[i], p.slot[i] = s.slot[i];
        for (int n = tid; n < p.N; n += 128) p.counts[n] = s.cnt[n];
        if (tid == 0)
            *p.aux = (float)(((s.aux[0] + s.aux[1]) + (s.aux[2] + s.aux[3])) * (double)p.N / ((double)p.T * p.T));
    }
    return true;
}

__device__ __forceinline__ int32_t atom_add_acq_rel_gpu(int32_t *p, int32_t v) {
    int32_t old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

}  // namespace switchmoe
