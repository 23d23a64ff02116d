// The whole layer for a few tokens (a decoding step): two kernels.
//
//   few_router   logits = W_r x (+ b), float32
//   few_experts  softmax, top-1 or top-2, slots, then for the experts that
//                were reached h = ReLU(W_in x) and o = W_out h, and
//                y = sum over the kept choices of gate * o
//
// With few tokens the layer is bound by reading the weights of the experts
// that the tokens reach (2 d F elements each) once.  So the second kernel is
// one persistent launch over both products: blocks claim items of work in
// order from a counter, all items of the first product before any of the
// second, and an item of the second product waits until the first product of
// its expert is complete (a counter per group).  Only running blocks hold
// claims and items of the first product wait for nothing, so the wait ends
// whatever else occupies the GPU; it is bounded all the same.  The block that
// finishes the last item of a tile of output rows forms y there, in a fixed
// order: no sum depends on the order in which blocks finish.
//
// This file: the router and the CUDA-core form (float32 experts, and any
// with SWITCH_FLAG_SIMT_FFN).
#include <type_traits>

#include "few.cuh"

namespace switchmoe {
namespace {

// ---------------------------------------------------------------------------
// element loads
// ---------------------------------------------------------------------------
__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float *v) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// V consecutive elements (V * sizeof(T) bytes aligned to their size, 16 at most)
template <typename T, int V>
__device__ __forceinline__ void load_elems(const T *p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = Elem<T>::load(p, 0);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 a = reinterpret_cast<const float4 *>(p)[i];
            v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
        }
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const uint2 a = reinterpret_cast<const uint2 *>(p)[i];
            v[4 * i] = __uint_as_float(a.x << 16), v[4 * i + 1] = __uint_as_float(a.x & 0xffff0000u);
            v[4 * i + 2] = __uint_as_float(a.y << 16), v[4 * i + 3] = __uint_as_float(a.y & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) e4m3x4_to_float(reinterpret_cast<const uint32_t *>(p)[i], v + 4 * i);
    }
}

// ---------------------------------------------------------------------------
// router
// ---------------------------------------------------------------------------
// Four warps of 64 registers: a block fits beside one of the second kernel's on an SM, so that neither
// kernel has to wait for the other's last block.  (In a graph the second kernel's blocks start within
// 0.5 us of the last router's end and are past their wait after 0.8 us.)
constexpr int kRouterThreads = 128;

// Block (i, j): the logits of TE experts for TT tokens, the dot products
// spread over the block's threads, V elements each; sums in a fixed order.
template <typename X, int V, int TE, int TT>
__global__ void __launch_bounds__(kRouterThreads, 8)
    few_router_kernel(const FewArgs p, int zero_ints, int want_xmax) {
    __shared__ float red[kRouterThreads / 32][TE * TT];
    __shared__ uint32_t big[kRouterThreads / 32][TT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int e0 = blockIdx.x * TE, t0 = blockIdx.y * TT;
    pdl_launch_dependents();
    pdl_wait();  // x; and the call before this one may still use the workspace
    {  // the second kernel's counters and maxima, and the status word
        const int blocks = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
        int32_t *z = reinterpret_cast<int32_t *>(p.ctr);
        for (int i = me * kRouterThreads + tid; i < zero_ints; i += blocks * kRouterThreads) z[i] = 0;
        if (me == 0 && tid < (int)(sizeof(DeviceStatus) / 4)) reinterpret_cast<int32_t *>(p.status)[tid] = 0;
    }
    const X *x = static_cast<const X *>(p.x);
    const float *w[TE];
    const X *xr[TT];
#pragma unroll
    for (int e = 0; e < TE; ++e) w[e] = p.w_r + (int64_t)min(e0 + e, p.N - 1) * p.d;
#pragma unroll
    for (int t = 0; t < TT; ++t) xr[t] = x + (int64_t)min(t0 + t, p.T - 1) * p.d;
    float acc[TE][TT];
    uint32_t top[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        top[t] = 0;
#pragma unroll
        for (int e = 0; e < TE; ++e) acc[e][t] = 0.f;
    }
    // several steps' loads in flight: rows of W_r come from memory, 1 us away
#pragma unroll(TE * TT == 1 ? 8 : TE == 1 ? 2 : 1)
    for (int j = tid * V; j < p.d; j += kRouterThreads * V) {
        float wv[TE][V];
#pragma unroll
        for (int e = 0; e < TE; ++e) load_elems<float, V>(w[e] + j, wv[e]);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            float xv[V];
            load_elems<X, V>(xr[t] + j, xv);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                top[t] = max(top[t], __float_as_uint(xv[i]) & 0x7fffffffu);
#pragma unroll
                for (int e = 0; e < TE; ++e) acc[e][t] = fmaf(wv[e][i], xv[i], acc[e][t]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < TE; ++e)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            float a = acc[e][t];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
            if (lane == 0) red[warp][e * TT + t] = a;
        }
    if (want_xmax && blockIdx.x == 0) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const uint32_t b = __reduce_max_sync(0xffffffffu, top[t]);
            if (lane == 0) big[warp][t] = b;
        }
    }
    __syncthreads();
    if (tid < TE * TT) {
        const int e = e0 + tid / TT, t = t0 + tid % TT;
        if (e < p.N && t < p.T) {
            float a = 0.f;
#pragma unroll
            for (int w8 = 0; w8 < kRouterThreads / 32; ++w8) a += red[w8][tid];
            if (p.x_scale != nullptr) a *= p.x_scale[t];
            if (p.bias != nullptr) a += p.bias[e];
            p.logits[(int64_t)t * p.N + e] = a;
        }
    }
    if (want_xmax && blockIdx.x == 0 && tid < TT && t0 + tid < p.T) {
        uint32_t b = 0;
        for (int w8 = 0; w8 < kRouterThreads / 32; ++w8) b = max(b, big[w8][tid]);
        p.xmax[t0 + tid] = b;
    }
}

template <typename X, int V, int TE, int TT>
cudaError_t router_launch(const FewArgs &p, int zero_ints, int want_xmax, cudaStream_t stream) {
    return launch_kernel(few_router_kernel<X, V, TE, TT>, dim3((p.N + TE - 1) / TE, (p.T + TT - 1) / TT),
                         dim3(kRouterThreads), 0, stream, true, p, zero_ints, want_xmax);
}

template <typename X, int V>
cudaError_t router_typed(const FewArgs &p, int zero_ints, int want_xmax, cudaStream_t stream) {
    // one expert per block for the most blocks in flight; with many blocks four, so that a row of x serves four
    if (p.T == 1) return router_launch<X, V, 1, 1>(p, zero_ints, want_xmax, stream);
    if (p.N * ((p.T + 3) / 4) <= 1184) return router_launch<X, V, 1, 4>(p, zero_ints, want_xmax, stream);
    return router_launch<X, V, 4, 4>(p, zero_ints, want_xmax, stream);
}

// ---------------------------------------------------------------------------
// experts on CUDA cores
// ---------------------------------------------------------------------------
constexpr int kSimtThreads = 256;
constexpr int kSimtBlocks = 2;  // per SM
constexpr int kSimtWarps = kSimtThreads / 32;
constexpr int kSimtRows = 8;  // weight rows of a team

template <int TOK>
struct SimtShared {
    FewPlan plan;
    float red[kSimtWarps][kSimtRows * TOK];
    int item, go, last;
};

// v[0..7] of every lane summed over the warp: lane l (a multiple of 4) is left
// with the sum of v[l / 4].  Each exchange halves the values, so eight sums
// take 9 shuffles and not 40.
__device__ __forceinline__ float sum8(float (&v)[8], int lane) {
    float u[4], w[2];
    const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float away = h16 ? v[i] : v[4 + i], mine = h16 ? v[4 + i] : v[i];
        u[i] = mine + __shfl_xor_sync(0xffffffffu, away, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float away = h8 ? u[i] : u[2 + i], mine = h8 ? u[2 + i] : u[i];
        w[i] = mine + __shfl_xor_sync(0xffffffffu, away, 8);
    }
    float s = (h4 ? w[1] : w[0]) + __shfl_xor_sync(0xffffffffu, h4 ? w[0] : w[1], 4);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    return s + __shfl_xor_sync(0xffffffffu, s, 1);
}

// red[j * 8 + r] = sum_k w[r][k] x_j[k], x_j the row token[j] (or j) of `in`,
// over this warp's share of k (steps first, first + TEAM, ... of 32 V elements),
// for kSimtRows rows of weights and m <= TOK tokens; rows past `rows_left`
// repeat the last one.  U steps' weights are in flight together, about as many as
// the registers beside the accumulators hold (19 of the 20 forms spill 42 to 262
// bytes; only that of odd sizes, four tokens and long rows does not).
template <typename W, typename X, int V, int TOK, int TEAM>
__device__ __forceinline__ void simt_dots(const W *w, int rows_left, int K, const X *in, const int *token, int m,
                                          int pitch, int first, int lane, float *red) {
    float acc[TOK][kSimtRows];
#pragma unroll
    for (int j = 0; j < TOK; ++j)
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) acc[j][r] = 0.f;
    constexpr int kStride = TEAM * 32 * V, U = TOK == 4 ? (V == 1 ? 6 : 2) : (V == 1 ? 4 : 1);
    for (int k0 = (first * 32 + lane) * V; k0 < K; k0 += U * kStride) {
        float wv[U][kSimtRows][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < kSimtRows; ++r) {
                const int k = k0 + u * kStride;
                if (u == 0 || k < K) {
                    load_elems<W, V>(w + (uint32_t)(min(r, rows_left - 1) * K + k), wv[u][r]);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) wv[u][r][i] = 0.f;
                }
            }
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            if (j >= m) break;
            const X *x = in + (int64_t)(token != nullptr ? token[j] : j) * pitch;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * kStride;
                if (u == 0 || k < K) {
                    float xv[V];
                    load_elems<X, V>(x + k, xv);
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int r = 0; r < kSimtRows; ++r) acc[j][r] = fmaf(wv[u][r][i], xv[i], acc[j][r]);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
        if (j >= m) break;
        const float s = sum8(acc[j], lane);
        if ((lane & 3) == 0) red[j * kSimtRows + (lane >> 2)] = s;
    }
}

// A block takes an item, for up to TOK tokens: 8 weight rows of one expert,
// their length dealt out to its 8 warps; 64 rows, 8 to a warp, where the rows
// are at most two steps long (20 tokens of 72 x 1284, 248 experts: 23 us, with 8
// rows 40 us; on long rows warps of their own measured slower, their x rows
// coming eight times as often).
template <int V>
__device__ __forceinline__ int simt_team(int K) {
    return K <= 64 * V ? 1 : kSimtWarps;
}

// V: elements that a lane takes of a weight row at a time.
// SHORT: W_in's or W_out's rows are (a kernel of its own: the other one's registers are all taken).
template <typename W, typename X, int V, int TOK, bool SHORT>
__global__ void __launch_bounds__(kSimtThreads, kSimtBlocks) few_experts_simt_kernel(const FewArgs p) {
    __shared__ SimtShared<TOK> s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();  // the logits and the zeroed counters
    int next = 0;
    if (tid == 0) next = atomicAdd(&p.ctr->claim, 1);
    few_plan(p, s.plan, TOK, kSimtThreads);
    const int team_h = SHORT ? simt_team<V>(p.d) : kSimtWarps, team_o = SHORT ? simt_team<V>(p.F) : kSimtWarps;
    const int rows_h = kSimtRows * kSimtWarps / team_h, rows_o = kSimtRows * kSimtWarps / team_o;  // of an item
    const int tiles_h = (p.F + rows_h - 1) / rows_h, tiles_o = (p.d + rows_o - 1) / rows_o;
    const int groups = s.plan.groups, items_h = groups * tiles_h, items = items_h + groups * tiles_o;
    bool gates = false;
    for (;;) {
        if (tid == 0) {
            s.item = next;
            if (next < items) next = atomicAdd(&p.ctr->claim, 1);  // runs while this item is computed
        }
        __syncthreads();
        const int item = s.item;
        if (!gates && item >= items_h) {  // between the products, when the first one's last parts are under way
            gates = true;
            if (tid < 128)
                few_gates(p, s.plan, tid, blockIdx.x == 0, [] {
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    return true;
                });
        }
        if (item >= items) break;
        if (item >= items_h) {
            if (tid == 0) s.go = wait_counter_geq(&p.ctr->done[(item - items_h) % groups], tiles_h, p.status, 71);
            __syncthreads();
            if (!s.go) break;
        }
        const bool second = item >= items_h;
        const int r0 = second ? item - items_h : item, q0 = r0 / (second ? groups : tiles_h);
        const int rest = r0 - q0 * (second ? groups : tiles_h);
        const int g = second ? rest : q0, tile = second ? q0 : rest;
        const int e = s.plan.g_expert[g], a0 = s.plan.g_first[g], m = s.plan.g_size[g];
        const int team = SHORT ? (second ? team_o : team_h) : kSimtWarps;
        const int tall = SHORT ? (second ? rows_o : rows_h) : kSimtRows;
        const int row0 = tile * tall, rows = second ? p.d : p.F, K = second ? p.F : p.d;
        const int mine = row0 + warp / team * kSimtRows;  // this team's first row
        const W *w = static_cast<const W *>(second ? p.w_out : p.w_in) + ((int64_t)e * rows + mine) * K;
        const X *x = static_cast<const X *>(p.x);
        const float *h = p.h + (int64_t)a0 * p.F;
        const int *list = s.plan.token + a0;
        float *red = s.red[warp];
        if (!SHORT || team == kSimtWarps) {
            if (second) simt_dots<W, float, V, TOK, kSimtWarps>(w, rows - mine, K, h, nullptr, m, K, warp, lane, red);
            else simt_dots<W, X, V, TOK, kSimtWarps>(w, rows - mine, K, x, list, m, K, warp, lane, red);
        } else if (mine < rows) {
            if (second) simt_dots<W, float, V, TOK, 1>(w, rows - mine, K, h, nullptr, m, K, 0, lane, red);
            else simt_dots<W, X, V, TOK, 1>(w, rows - mine, K, x, list, m, K, 0, lane, red);
        }
        __syncthreads();
        for (int i = tid; i < tall * m; i += kSimtThreads) {
            const int j = i / tall, r = i - j * tall, row = row0 + r;
            if (row < rows) {
                float v = 0.f;
#pragma unroll SHORT ? 1 : kSimtWarps
                for (int q = 0; q < team; ++q) v += s.red[r / kSimtRows * team + q][j * kSimtRows + r % kSimtRows];
                if (second) {
                    if (p.w_out_scale != nullptr) v *= p.w_out_scale[(int64_t)e * p.d + row];
                    p.o[(int64_t)(a0 + j) * p.d + row] = v;
                } else {
                    if (p.w_in_scale != nullptr) v *= p.w_in_scale[(int64_t)e * p.F + row];
                    if (p.x_scale != nullptr) v *= p.x_scale[s.plan.token[a0 + j]];
                    p.h[(int64_t)(a0 + j) * p.F + row] = v < 0.f ? 0.f : v;  // NaN stays NaN
                }
            }
        }
        __syncthreads();
        if (tid == 0) {
            if (second) s.last = atom_add_acq_rel_gpu(&p.ctr->tile[tile], 1) == groups - 1;
            else red_release_add_gpu(&p.ctr->done[g], 1);
        }
        if (second) {
            __syncthreads();
            if (s.last) {  // y of the tile's rows for every token
                for (int i = tid; i < p.T * tall; i += kSimtThreads) {
                    const int t = i / tall, row = row0 + i - t * tall;
                    if (row >= p.d) continue;
                    float y = 0.f;
                    for (int c = 0; c < p.k; ++c) {
                        const int a = s.plan.pos[t * p.k + c];
                        if (a >= 0) y += s.plan.gate[t * p.k + c] * __ldcg(p.o + (int64_t)a * p.d + row);
                    }
                    p.y[(int64_t)t * p.d + row] = y;
                }
            }
        }
    }
}

template <typename W, typename X, int V>
cudaError_t experts_simt(const FewArgs &p, cudaStream_t stream) {
    // Few pairs: groups of up to 4 tokens, whose accumulators leave registers for more weights in flight (2 tokens
    // of 4096 x 10000: 113 us, with 8 117 us); many: 8, so that weights are read for more tokens at a time (32
    // tokens top-2 of 1024 x 2048: 106 us, with 4 121 us).
    const bool few = p.T * p.k <= 16;
    const bool brief = p.d <= 64 * V || p.F <= 64 * V;
    auto *kernel = few ? (brief ? few_experts_simt_kernel<W, X, V, 4, true> : few_experts_simt_kernel<W, X, V, 4, false>)
                       : (brief ? few_experts_simt_kernel<W, X, V, 8, true> : few_experts_simt_kernel<W, X, V, 8, false>);
    return launch_kernel(kernel, dim3(device_sm_count() * kSimtBlocks), dim3(kSimtThreads), 0, stream, true, p);
}

}  // namespace

namespace {

// Parts that the length of a product may be cut into: enough to give every SM
// work when few pairs keep few tiles, and 512 rows of partial sums at most.
int few_max_splits(int64_t pairs) {
    const int64_t s = pairs > 0 ? 512 / pairs : 16;
    return (int)(s > 16 ? 16 : s);
}

struct FewSections {
    size_t status, ctr, hmax, parts, xmax, logits, h, o, total;
};
FewSections few_layout(const switch_dims_t &d, int top_k) {
    const size_t A = (size_t)d.T * top_k, S = (size_t)few_max_splits((int64_t)A);
    FewSections s{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) / 256 * 256;
        return at;
    };
    s.status = take(sizeof(DeviceStatus));
    s.ctr = off;  // the counters, hmax and parts right behind one another are zeroed as one range
    off += sizeof(FewCounters);
    s.hmax = off;
    off += S * A * 4;
    s.parts = off;
    take((size_t)((d.d_model + 127) / 128) * 4 * (size_t)d.T * 4);
    off = (off + 255) / 256 * 256;
    s.xmax = take((size_t)d.T * 4);
    s.logits = take((size_t)d.T * d.num_experts * 4);
    s.h = take(S * A * (size_t)d.d_ff * 4);
    s.o = take(S * A * (size_t)d.d_model * 4);
    s.total = off;
    return s;
}

}  // namespace

size_t few_workspace_bytes(const switch_dims_t &dims, int top_k) { return few_layout(dims, top_k).total; }

cudaError_t launch_layer_few(const switch_dims_t &dims, int x_dtype, FewArgs &p, void *workspace,
                             cudaStream_t stream) {
    const FewSections s = few_layout(dims, p.k);
    uint8_t *b = static_cast<uint8_t *>(workspace);
    p.status = reinterpret_cast<DeviceStatus *>(b + s.status);
    p.ctr = reinterpret_cast<FewCounters *>(b + s.ctr);
    p.hmax = reinterpret_cast<uint32_t *>(b + s.hmax);
    p.parts = reinterpret_cast<int32_t *>(b + s.parts);
    p.xmax = reinterpret_cast<uint32_t *>(b + s.xmax);
    p.logits = reinterpret_cast<float *>(b + s.logits);
    p.h = reinterpret_cast<float *>(b + s.h);
    p.o = reinterpret_cast<float *>(b + s.o);
    if (p.T == 0) {
        cudaError_t err = cudaMemsetAsync(p.status, 0, sizeof(DeviceStatus), stream);
        if (err == cudaSuccess) err = cudaMemsetAsync(p.counts, 0, (size_t)p.N * 4, stream);
        return err == cudaSuccess ? cudaMemsetAsync(p.aux, 0, 4, stream) : err;
    }
    const int splits = few_max_splits(p.T * p.k);
    const bool tensor_cores = dims.dtype != SWITCH_F32 && !(dims.flags & SWITCH_FLAG_SIMT_FFN);
    const bool cut_x = tensor_cores && dims.dtype == SWITCH_E4M3 && x_dtype == SWITCH_BF16;
    const int zero_ints =
        (int)(sizeof(FewCounters) / 4) + (tensor_cores ? splits * p.T * p.k + (p.d + 127) / 128 * 4 * p.T : 0);
    const cudaError_t err = launch_few_router(p, x_dtype, zero_ints, cut_x, stream);
    if (err != cudaSuccess) return err;
    return tensor_cores ? launch_few_experts_tc(p, dims.dtype, x_dtype, splits, stream)
                        : launch_few_experts_simt(p, dims.dtype, x_dtype, stream);
}

cudaError_t launch_few_router(const FewArgs &p, int x_dtype, int zero_ints, bool want_xmax, cudaStream_t stream) {
    launch_begin(K_FEW_ROUTER, stream);
    cudaError_t err;
    if (x_dtype == SWITCH_BF16) err = router_typed<__nv_bfloat16, 4>(p, zero_ints, want_xmax, stream);
    else if (x_dtype == SWITCH_E4M3) err = router_typed<uint8_t, 4>(p, zero_ints, want_xmax, stream);
    else if (p.d % 4 == 0) err = router_typed<float, 4>(p, zero_ints, want_xmax, stream);
    else err = router_typed<float, 1>(p, zero_ints, want_xmax, stream);
    launch_end(stream);
    return err;
}

cudaError_t launch_few_experts_simt(const FewArgs &p, int w_dtype, int x_dtype, cudaStream_t stream) {
    launch_begin(K_FEW_EXPERTS_SIMT, stream);
    cudaError_t err;
    if (w_dtype == SWITCH_BF16) err = experts_simt<__nv_bfloat16, __nv_bfloat16, 4>(p, stream);
    else if (w_dtype == SWITCH_E4M3 && x_dtype == SWITCH_E4M3) err = experts_simt<uint8_t, uint8_t, 4>(p, stream);
    else if (w_dtype == SWITCH_E4M3) err = experts_simt<uint8_t, __nv_bfloat16, 4>(p, stream);
    else if (p.d % 4 == 0 && p.F % 4 == 0) err = experts_simt<float, float, 4>(p, stream);
    else err = experts_simt<float, float, 1>(p, stream);
    launch_end(stream);
    return err;
}

}  // namespace switchmoe
