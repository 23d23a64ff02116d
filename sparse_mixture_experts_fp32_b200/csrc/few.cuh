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
    uint32_t *hmax;    // [kFewMaxSplit][A] bits of max |partial sum| of a pair's hidden row
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
    uint32_t order[kFewMaxA / 4];  // expert of every pair, a byte each, first choices before second ones
    float top[kFewMaxT], total[kFewMaxT];  // softmax maximum and sum of each token
    int cnt[kFewMaxN], base[kFewMaxN];
    int g_expert[kFewMaxA], g_first[kFewMaxA], g_size[kFewMaxA];
    int groups, largest;     // groups; positions of the largest one
};

// Every thread of a block of `threads` (a multiple of 32, at least 128) calls
// this; block 0 also writes the call's routing outputs.  T and N are small
// (64 x 256 logits at most), so that every block deciding for itself costs less
// than another kernel or a grid-wide wait would.
__device__ inline void few_plan(const FewArgs &p, FewPlan &s, int group_max, int threads) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = threads >> 5;
    const int A = p.T * p.k;
    for (int n = tid; n < p.N; n += threads) s.cnt[n] = 0;
    for (int i = tid; i < kFewMaxA / 4; i += threads) s.order[i] = 0;
    __syncthreads();
    for (int t = warp; t < p.T; t += warps) {
        float v[kFewMaxN / 32];
#pragma unroll
        for (int i = 0; i < kFewMaxN / 32; ++i) {
            const int n = 32 * i + lane;
            v[i] = n < p.N ? __ldcg(p.logits + (int64_t)t * p.N + n) : -INFINITY;
        }
        int first = -1;
        float top = 0.f;
        for (int c = 0; c < p.k; ++c) {
            float best = -INFINITY;
            int at = INT32_MAX;
#pragma unroll
            for (int i = 0; i < kFewMaxN / 32; ++i) {
                const int n = 32 * i + lane;
                if (n < p.N && n != first && (v[i] > best || (v[i] == best && n < at))) best = v[i], at = n;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float b = __shfl_xor_sync(0xffffffffu, best, o);
                const int a = __shfl_xor_sync(0xffffffffu, at, o);
                if (b > best || (b == best && a < at)) best = b, at = a;
            }
            if (at == INT32_MAX) at = first == 0 ? 1 : 0;  // no logit compares (NaN): any expert, with a NaN gate
            if (c == 0) {
                top = best;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kFewMaxN / 32; ++i)
                    if (32 * i + lane < p.N) sum += expf(v[i] - top);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0) s.top[t] = top, s.total[t] = sum;
                first = at;
                __syncwarp();
            }
            if (lane == 0) {
                s.expert[t * p.k + c] = at;
                s.gate[t * p.k + c] = expf(best - top) / s.total[t];
                reinterpret_cast<uint8_t *>(s.order)[c * p.T + t] = (uint8_t)at;
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < A; i += threads) {  // rank among the pairs of its expert; first choices come first
        const int t = i % p.T, c = i / p.T, e = s.expert[t * p.k + c];
        const uint32_t four = (uint32_t)e * 0x01010101u;
        int rank = 0;
        for (int w = 0; w < i / 4; ++w) rank += __popc(__vcmpeq4(s.order[w], four)) >> 3;
        if (i & 3) rank += __popc(__vcmpeq4(s.order[i >> 2], four) & ((1u << (8 * (i & 3))) - 1u)) >> 3;
        s.slot[t * p.k + c] = rank < p.C ? rank : -1;
        atomicAdd(&s.cnt[e], 1);
    }
    __syncthreads();
    if (warp == 0) {
        int pairs = 0, groups = 0, largest = 0;
        for (int n0 = 0; n0 < p.N; n0 += 32) {
            const int n = n0 + lane;
            const int kept = n < p.N ? min(s.cnt[n], p.C) : 0;
            const int mine = (kept + group_max - 1) / group_max;
            int a = kept, g = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int ua = __shfl_up_sync(0xffffffffu, a, o), ug = __shfl_up_sync(0xffffffffu, g, o);
                if (lane >= o) a += ua, g += ug;
            }
            if (n < p.N) s.base[n] = pairs + a - kept;
            for (int j = 0; j < mine; ++j) {
                const int at = groups + g - mine + j;
                s.g_expert[at] = n;
                s.g_first[at] = pairs + a - kept + j * group_max;
                s.g_size[at] = min(group_max, kept - j * group_max);
            }
            largest = max(largest, min(group_max, kept));
            pairs += __shfl_sync(0xffffffffu, a, 31);
            groups += __shfl_sync(0xffffffffu, g, 31);
        }
        largest = __reduce_max_sync(0xffffffffu, largest);
        if (lane == 0) s.groups = groups, s.largest = largest;
    }
    __syncthreads();
    for (int i = tid; i < A; i += threads) {
        const int at = s.slot[i] < 0 ? -1 : s.base[s.expert[i]] + s.slot[i];
        s.pos[i] = at;
        if (at >= 0) s.token[at] = i / p.k;
    }
    if (blockIdx.x == 0) {
        for (int i = tid; i < A; i += threads) p.expert[i] = s.expert[i], p.gate[i] = s.gate[i], p.slot[i] = s.slot[i];
        for (int n = tid; n < p.N; n += threads) p.counts[n] = s.cnt[n];
        if (warp == 0) {  // aux = N sum_n (first choices of n / T) (mean_t p_n): float64, in a fixed order
            double sum = 0.0;
            for (int n = lane; n < p.N; n += 32) {
                double prob = 0.0;
                int f = 0;
                for (int t = 0; t < p.T; ++t) {
                    prob += (double)(expf(__ldcg(p.logits + (int64_t)t * p.N + n) - s.top[t]) / s.total[t]);
                    f += s.expert[t * p.k] == n;
                }
                sum += (double)f * prob;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) *p.aux = (float)(sum * (double)p.N / ((double)p.T * (double)p.T));
        }
    }
    __syncthreads();
}

// y of the output rows [row0, row0 + rows) for all tokens, by the block that
// finished the rows' last item; `threads` threads call it (tid < threads).
__device__ inline void few_combine(const FewArgs &p, const FewPlan &s, int splits, int A, int row0, int rows, int tid,
                                   int threads) {
    for (int i = tid; i < p.T * rows; i += threads) {
        const int t = i / rows, row = row0 + i % rows;
        float y = 0.f;
        for (int c = 0; c < p.k; ++c) {
            const int a = s.pos[t * p.k + c];
            if (a < 0) continue;
            float o = 0.f;
            for (int q = 0; q < splits; ++q) o += __ldcg(p.o + ((int64_t)q * A + a) * p.d + row);
            y += s.gate[t * p.k + c] * o;
        }
        p.y[(int64_t)t * p.d + row] = y;
    }
}

}  // namespace switchmoe
