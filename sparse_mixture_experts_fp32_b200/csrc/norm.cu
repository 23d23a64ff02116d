// What stands before the layer: the residual's addition with its
// root-mean-square norm, that norm's gradient, and rows in 8 bits with scales.
//
//   s      = residual + delta             rounded once to the residual's type
//   rstd   = 1 / sqrt(mean_j s_j^2 + eps)
//   v_j    = s_j rstd weight_j            rounded once to the output's type, or
//   scale  = max_j |v_j| / 448,  q_j = e4m3(v_j / scale)
// and, for an upstream gradient g of v and dsum of s,
//   ds_j      = dsum_j + rstd (g_j w_j - s_j rstd m),  m = mean_j (g_j w_j s_j rstd)
//   dweight_j = sum over rows of g_j s_j rstd
// (the gradient goes through the rounding of s as through the identity).
//
// All of them are bound by memory: a row is read once into registers, reduced
// there and written once.  A group of `tpr` threads holds a row, 8 elements (16
// or 32 bytes) per thread; widths that are no multiple of 8 take the same
// kernels with one element per thread and step, since their rows start at any
// alignment (four steps where a block can hold the row so: 65536 x 257 to 8
// bits 84 us, eight steps 102 us).  Blocks live for one row group (a loop over rows that loads the
// next one early measured 20 % slower: 237 us); only the gradient, which keeps
// column sums, loops.  Sums and the norm are float32 (8 terms per thread, then
// a tree); the maxima are taken on the bit patterns of |v|, whose order is that
// of the values and puts NaN on top, so that a row with a NaN gets a NaN scale.
//
// Measured on a B200 (copy bandwidth 6549 GB/s): 131072 x 1024 bfloat16 +
// float32 -> bfloat16 194 us (6.9 TB/s), its gradient 304 us (6.2 TB/s);
// 8192 x 768 float32 + float32 -> 8 bits 16.5 us (5.0 TB/s); 131072 x 1024
// bfloat16 to 8 bits 87 us (4.6 TB/s).
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace switchmoe {
namespace {

constexpr float kE4m3Max = 448.f;
#ifndef QI
#define QI 4
#endif
struct None {};  // no delta

template <typename T, int VEC>
__device__ __forceinline__ void load_row(const T *p, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = Elem<T>::load(p, 0);
    } else if constexpr (sizeof(T) == 4) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_row(T *p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        Elem<T>::store(p, 0, v[0]);
    } else if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
}

template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        *p = (uint8_t)__nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi =
                __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

// Sum (or maximum of unsigned) over the `tpr` threads of a row; every thread
// of the block calls it.  `part` has a slot per warp of the block, and a block
// uses another `part` for its next sum (or the one before its last one).
__device__ __forceinline__ float row_sum(float v, int tpr, float *part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr == 32) return v;
    const int tid = threadIdx.y * tpr + threadIdx.x, warp = tid >> 5, warps = tpr >> 5, w0 = threadIdx.y * warps;
    if ((tid & 31) == 0) part[warp] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += part[w0 + w];
    return s;
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, int tpr, float *part) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (tpr == 32) return v;
    uint32_t *p = reinterpret_cast<uint32_t *>(part);
    const int tid = threadIdx.y * tpr + threadIdx.x, warp = tid >> 5, warps = tpr >> 5, w0 = threadIdx.y * warps;
    if ((tid & 31) == 0) p[warp] = v;
    __syncthreads();
    uint32_t s = 0;
    for (int w = 0; w < warps; ++w) s = max(s, p[w0 + w]);
    return s;
}

// e4m3's rounding of v / s is that of t = v * (1 / s), which is within 2 units in the last place of the
// quotient, unless t is as close to the middle between two e4m3 values: in the normal range those have
// the 20 low bits 0x80000.  Such t, and the few below the normal range, are divided for.  (A division for
// every element bounds the kernel: 131072 x 1024 bfloat16 took 116 us with it, 90 us with this.)
struct Doubt {
    uint32_t middle = 0xffffffffu, small = 0xffffffffu;  // least distances (as unsigned numbers) over a thread's values
    __device__ __forceinline__ void see(float t) {
        const uint32_t b = __float_as_uint(t);
        middle = min(middle, (b & 0xfffffu) - 0x7fff8u);
        small = min(small, (b << 1) - 1u);  // a zero is not small
    }
    __device__ __forceinline__ bool any() const { return middle <= 0x10u || small < 0x78ffffffu; }  // |t| < 2^-6
};

// Scale of a row whose largest |v| has the bits `top`, and the rounding of its values.
struct Quantizer {
    float s, inv;
    bool tiny;  // 1 / s may overflow
    __device__ explicit Quantizer(uint32_t top) {
        s = __fdiv_rn(__uint_as_float(top), kE4m3Max);
        inv = __frcp_rn(s);
        tiny = s < 1e-30f;
    }
    template <int VEC>
    __device__ __forceinline__ void store(uint8_t *q, const float (&v)[VEC]) const {
        float u[VEC];
        Doubt doubt;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            u[k] = v[k] * inv;
            doubt.see(u[k]);
        }
        if (tiny || doubt.any()) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) u[k] = s == 0.f ? 0.f : __fdiv_rn(v[k], s);  // a row of zeros: scale 0
        }
        store_e4m3<VEC>(q, u);
    }
};

// The row in registers -> e4m3 and its scale.
template <int VEC, int ITERS>
__device__ __forceinline__ void quantize_row(const float (&v)[ITERS][VEC], int d, int tpr, float *part, bool live,
                                             uint8_t *q, float *scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) top = max(top, __float_as_uint(v[i][k]) & 0x7fffffffu);
    const Quantizer z(row_max(top, tpr, part));
    if (!live) return;
    if (threadIdx.x == 0) *scale = z.s;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int j = (i * tpr + (int)threadIdx.x) * VEC;
        if (j < d) z.store<VEC>(q + j, v[i]);
    }
}

template <typename R, typename D, typename O, int VEC, int ITERS>
__global__ void __launch_bounds__(1024)
    norm_fwd_kernel(const R *residual, const D *delta, const float *__restrict__ weight, R *sum, O *out,
                    float *__restrict__ scale, float *__restrict__ rstd, int64_t T, int d, float eps) {
    constexpr bool kDelta = !std::is_same<D, None>::value;
    __shared__ float part[2][32];
    const int tpr = blockDim.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < T;
    const int64_t row = live ? t * d : 0;
    float s[ITERS][VEC];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int j = (i * tpr + (int)threadIdx.x) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[i][k] = 0.f;
        if (live && j < d) {
            load_row<R, VEC>(residual + row + j, s[i]);
            if constexpr (kDelta) {
                float a[VEC];
                load_row<D, VEC>(delta + row + j, a);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    s[i][k] += a[k];
                    // the sum is normalised as it is stored: the backward pass reads the stored one
                    if constexpr (sizeof(R) == 2) s[i][k] = bf16_bits_to_float(float_to_bf16_bits(s[i][k]));
                }
            }
        }
    }
    if constexpr (kDelta) {
        if (sum != nullptr) {
#pragma unroll
            for (int i = 0; i < ITERS; ++i) {
                const int j = (i * tpr + (int)threadIdx.x) * VEC;
                if (live && j < d) store_row<R, VEC>(sum + row + j, s[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) ss = fmaf(s[i][k], s[i][k], ss);
    const float r = __frcp_rn(__fsqrt_rn(row_sum(ss, tpr, part[0]) / (float)d + eps));
    if (live && threadIdx.x == 0 && rstd != nullptr) rstd[t] = r;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int j = (i * tpr + (int)threadIdx.x) * VEC;
        if (j >= d) break;
        float w[VEC];
        load_row<float, VEC>(weight + j, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[i][k] = s[i][k] * r * w[k];
    }
    if constexpr (sizeof(O) == 1) {
        quantize_row<VEC, ITERS>(s, d, tpr, part[1], live, reinterpret_cast<uint8_t *>(out) + row, scale + t);
    } else {
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
            if (live && j < d) store_row<O, VEC>(out + row + j, s[i]);
        }
    }
}

template <typename R, int VEC, int ITERS, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 && VEC == 8 && sizeof(R) == 2 ? 6 : 1)
    quantize_rows_kernel(const R *__restrict__ x, uint8_t *__restrict__ q, float *__restrict__ scale, int64_t rows,
                         int cols) {
    __shared__ float part[32];
    const int tpr = blockDim.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < rows;
    const int64_t row = live ? t * cols : 0;
    if constexpr (VEC == 8 && sizeof(R) == 2) {
        // the row stays in its 16 bits until it is rounded: half the registers, twice the rows in flight
        uint4 raw[ITERS];
        uint32_t top2 = 0;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
            raw[i] = live && j < cols ? *reinterpret_cast<const uint4 *>(x + row + j) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            top2 = __vmaxu2(top2, __vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu));
            top2 = __vmaxu2(top2, __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu));
        }
        const Quantizer z(row_max(max(top2 << 16, top2 & 0xffff0000u), tpr, part));
        if (!live) return;
        if (threadIdx.x == 0) scale[t] = z.s;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
            if (j >= cols) break;
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            float v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            z.store<8>(q + row + j, v);
        }
    } else {
        float v[ITERS][VEC];
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[i][k] = 0.f;
            if (live && j < cols) load_row<R, VEC>(x + row + j, v[i]);
        }
        quantize_row<VEC, ITERS>(v, cols, tpr, part, live, q + row, scale + t);
    }
}

// Each block takes every gridDim-th group of blockDim.y rows, keeps the
// columns' sums of g * s * rstd of its rows in registers and leaves their sum
// over its rows in part_dw[block]; dweight_kernel adds the blocks in order.
// A thread holds 8 elements of a row, so that enough blocks fit on an SM to
// keep memory busy (32 elements: 600 us at 131072 x 1024, 8: 304 us), and loads
// the next row's while this one's sum is formed.
template <typename R, int VEC, int ITERS, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? (VEC == 8 ? 4 : 2) : 1)
    norm_bwd_kernel(const R *__restrict__ sum, const float *__restrict__ weight, const float *__restrict__ rstd,
                    const float *dout, const float *dsum, float *dres, float *__restrict__ part_dw, int64_t T, int d) {
    extern __shared__ float columns[];  // [blockDim.y][d] when a block holds several rows
    __shared__ float part[2][32];
    const int tpr = blockDim.x;
    float w[ITERS][VEC], dw[ITERS][VEC];
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int j = (i * tpr + (int)threadIdx.x) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[i][k] = dw[i][k] = 0.f;
        if (j < d) load_row<float, VEC>(weight + j, w[i]);
    }
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    float h[ITERS][VEC], g[ITERS][VEC];
    float r = 0.f;
    auto load = [&](int64_t t) {
        const bool live = t < T;
        r = live ? rstd[t] : 0.f;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
#pragma unroll
            for (int k = 0; k < VEC; ++k) h[i][k] = g[i][k] = 0.f;
            if (live && j < d) {
                load_row<R, VEC>(sum + t * d + j, h[i]);
                load_row<float, VEC>(dout + t * d + j, g[i]);
            }
        }
    };
    load((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * blockDim.y; t0 < T; t0 += step) {
        const int64_t t = t0 + threadIdx.y;
        const bool live = t < T;
        const float rt = r;
        float u[ITERS][VEC], b[ITERS][VEC];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
#pragma unroll
            for (int k = 0; k < VEC; ++k) u[i][k] = 0.f;
            if (live && j < d && dsum != nullptr) load_row<float, VEC>(dsum + t * d + j, u[i]);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float hat = h[i][k] * rt;
                dw[i][k] = fmaf(g[i][k], hat, dw[i][k]);
                const float gw = g[i][k] * w[i][k];
                dot = fmaf(gw, hat, dot);
                u[i][k] = fmaf(rt, gw, u[i][k]);
                b[i][k] = rt * hat;
            }
        }
        load(t + step);
        const float m = row_sum(dot, tpr, part[turn]) / (float)d;
        turn ^= 1;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
            if (live && j < d) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) u[i][k] = fmaf(-m, b[i][k], u[i][k]);
                store_row<float, VEC>(dres + t * d + j, u[i]);
            }
        }
    }
    float *mine = part_dw + (int64_t)blockIdx.x * d;
    if (blockDim.y == 1) {
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
            if (j < d) store_row<float, VEC>(mine + j, dw[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (j + k < d) columns[threadIdx.y * d + j + k] = dw[i][k];
        }
        __syncthreads();
        const int threads = blockDim.x * blockDim.y;
        for (int j = threadIdx.y * tpr + threadIdx.x; j < d; j += threads) {
            float a = 0.f;
            for (int y = 0; y < (int)blockDim.y; ++y) a += columns[y * d + j];
            mine[j] = a;
        }
    }
    pdl_launch_dependents();
}

// dweight_j = sum over the blocks: 32 columns x 32 interleaved shares of the
// blocks per block, joined in a fixed order in float64.
constexpr int kShares = 32;
__global__ void __launch_bounds__(32 * kShares)
    dweight_kernel(const float *__restrict__ part, int blocks, int d, float *__restrict__ dweight) {
    __shared__ double acc[kShares][32];
    const int j = blockIdx.x * 32 + threadIdx.x;
    pdl_wait();
    double a = 0.0;
    if (j < d)
#pragma unroll 8
        for (int b = threadIdx.y; b < blocks; b += kShares) a += (double)part[(int64_t)b * d + j];
    acc[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && j < d) {
        for (int y = 1; y < kShares; ++y) a += acc[y][threadIdx.x];
        dweight[j] = (float)a;
    }
}

// Threads per row and rows per block for `iters` steps per thread.  Rows that a
// warp holds need no barrier and come eight to a block; other blocks have 128
// threads or one row, so that few rows wait for one another at a barrier
// (the gradient, 131072 x 1024: 256 threads 318 us, 128 threads 304 us).
struct RowShape {
    int tpr, rows, iters;
};
RowShape shape_of(int n, int iters) {
    const int tpr = (n + 32 * iters - 1) / (32 * iters) * 32;
    return {tpr, tpr == 32 ? 8 : tpr >= 128 ? 1 : 128 / tpr, iters};
}

template <typename R, typename D, typename O>
void norm_fwd_typed(const switch_norm_dims_t &n, const void *residual, const void *delta, const float *weight,
                    void *sum, void *out, float *scale, float *rstd, cudaStream_t stream) {
    const bool wide = n.d_model % 8 == 0;
    const RowShape s = wide ? shape_of(n.d_model / 8, 1) : shape_of(n.d_model, n.d_model <= 4096 ? 4 : 8);
    const dim3 grid((unsigned)((n.T + s.rows - 1) / s.rows)), block(s.tpr, s.rows);
#define SWITCH_NORM_FWD(V, I)                                                                                  \
    norm_fwd_kernel<R, D, O, V, I><<<grid, block, 0, stream>>>(                                                \
        static_cast<const R *>(residual), static_cast<const D *>(delta), weight, static_cast<R *>(sum),        \
        static_cast<O *>(out), scale, rstd, n.T, n.d_model, n.eps)
    if (wide) SWITCH_NORM_FWD(8, 1);
    else if (s.iters == 4) SWITCH_NORM_FWD(1, 4);
    else SWITCH_NORM_FWD(1, 8);
#undef SWITCH_NORM_FWD
}

template <typename R, typename D>
void norm_fwd_out(const switch_norm_dims_t &n, const void *residual, const void *delta, const float *weight, void *sum,
                  void *out, float *scale, float *rstd, cudaStream_t stream) {
    if (n.out_dtype == SWITCH_F32) norm_fwd_typed<R, D, float>(n, residual, delta, weight, sum, out, scale, rstd, stream);
    else if (n.out_dtype == SWITCH_BF16)
        norm_fwd_typed<R, D, __nv_bfloat16>(n, residual, delta, weight, sum, out, scale, rstd, stream);
    else norm_fwd_typed<R, D, uint8_t>(n, residual, delta, weight, sum, out, scale, rstd, stream);
}

template <typename R>
void norm_fwd_delta(const switch_norm_dims_t &n, const void *residual, const void *delta, const float *weight,
                    void *sum, void *out, float *scale, float *rstd, cudaStream_t stream) {
    if (delta == nullptr) norm_fwd_out<R, None>(n, residual, nullptr, weight, nullptr, out, scale, rstd, stream);
    else if (n.delta_dtype == SWITCH_F32) norm_fwd_out<R, float>(n, residual, delta, weight, sum, out, scale, rstd, stream);
    else norm_fwd_out<R, __nv_bfloat16>(n, residual, delta, weight, sum, out, scale, rstd, stream);
}

template <typename R>
void norm_bwd_typed(const switch_norm_dims_t &n, const RowShape &s, int blocks, const void *sum, const float *weight,
                    const float *rstd, const float *dout, const float *dsum, float *dres, float *part,
                    cudaStream_t stream) {
    const dim3 block(s.tpr, s.rows);
    const size_t smem = s.rows > 1 ? (size_t)s.rows * n.d_model * sizeof(float) : 0;
#define SWITCH_NORM_BWD(V, I, N)                                                                                  \
    norm_bwd_kernel<R, V, I, N><<<blocks, block, smem, stream>>>(static_cast<const R *>(sum), weight, rstd, dout, \
                                                                 dsum, dres, part, n.T, n.d_model)
    if (s.tpr <= 256) {
        if (n.d_model % 8 == 0) SWITCH_NORM_BWD(8, 1, 256);
        else SWITCH_NORM_BWD(1, 8, 256);
    } else {
        if (n.d_model % 8 == 0) SWITCH_NORM_BWD(8, 1, 1024);
        else SWITCH_NORM_BWD(1, 8, 1024);
    }
#undef SWITCH_NORM_BWD
}

template <typename R>
void quantize_typed(int64_t rows, int cols, const void *x, void *q, float *scale, cudaStream_t stream) {
    // Four steps per thread, a row to a warp, once there are rows enough to fill the GPU with warps: 16384 x 1024
    // takes 15 us so and 19 us with one step, 4096 x 1024 6.2 us and 5.8 us.
    const bool wide = cols % 8 == 0, large = rows * (int64_t)cols > (1 << 23) || cols > 8192;
    const RowShape s = wide ? shape_of(cols / 8, large ? 4 : 1) : shape_of(cols, cols <= 4096 ? 4 : cols <= 8192 ? 8 : 32);
    const dim3 grid((unsigned)((rows + s.rows - 1) / s.rows)), block(s.tpr, s.rows);
#define SWITCH_QUANT(V, I, N)                                                                      \
    quantize_rows_kernel<R, V, I, N><<<grid, block, 0, stream>>>(static_cast<const R *>(x),        \
                                                                 static_cast<uint8_t *>(q), scale, rows, cols)
    if (wide && s.iters == 1) SWITCH_QUANT(8, 1, 1024);
    else if (wide && s.tpr <= 256) SWITCH_QUANT(8, 4, 256);
    else if (wide) SWITCH_QUANT(8, 4, 1024);
    else if (s.iters == 4) SWITCH_QUANT(1, 4, 1024);
    else if (s.iters == 8) SWITCH_QUANT(1, 8, 1024);
    else SWITCH_QUANT(1, 32, 1024);
#undef SWITCH_QUANT
}

RowShape bwd_shape(const switch_norm_dims_t &n) {
    return n.d_model % 8 == 0 ? shape_of(n.d_model / 8, 1) : shape_of(n.d_model, 8);
}

int bwd_blocks(const switch_norm_dims_t &n) {
    const RowShape s = bwd_shape(n);
    const int64_t groups = (n.T + s.rows - 1) / s.rows;
    // as many blocks as are resident: 64 registers a thread leave an SM 1024 threads (128 half as many)
    const int64_t most = (int64_t)kNormBwdSms * (n.d_model % 8 == 0 || s.tpr > 256 ? 1024 : 512) / (s.tpr * s.rows);
    return (int)(groups < most ? groups : most);
}

}  // namespace

size_t norm_workspace_bytes(const switch_norm_dims_t &n) {
    const size_t bytes = (size_t)bwd_blocks(n) * (size_t)n.d_model * sizeof(float);
    return bytes < 256 ? 256 : (bytes + 255) / 256 * 256;
}

cudaError_t launch_norm_fwd(const switch_norm_dims_t &n, const void *residual, const void *delta, const float *weight,
                            void *sum, void *out, float *scale, float *rstd, cudaStream_t stream) {
    if (n.T == 0) return cudaSuccess;
    launch_begin(K_NORM_FWD, stream);
    if (n.residual_dtype == SWITCH_F32) norm_fwd_delta<float>(n, residual, delta, weight, sum, out, scale, rstd, stream);
    else norm_fwd_delta<__nv_bfloat16>(n, residual, delta, weight, sum, out, scale, rstd, stream);
    const cudaError_t err = cudaGetLastError();
    launch_end(stream);
    return err;
}

cudaError_t launch_norm_bwd(const switch_norm_dims_t &n, const void *sum, const float *weight, const float *rstd,
                            const float *dout, const float *dsum, float *dres, float *dweight, void *workspace,
                            cudaStream_t stream) {
    if (n.T == 0) return cudaMemsetAsync(dweight, 0, (size_t)n.d_model * sizeof(float), stream);
    const RowShape s = bwd_shape(n);
    const int blocks = bwd_blocks(n);
    float *part = static_cast<float *>(workspace);
    launch_begin(K_NORM_BWD, stream);
    if (n.residual_dtype == SWITCH_F32) norm_bwd_typed<float>(n, s, blocks, sum, weight, rstd, dout, dsum, dres, part, stream);
    else norm_bwd_typed<__nv_bfloat16>(n, s, blocks, sum, weight, rstd, dout, dsum, dres, part, stream);
    cudaError_t err = cudaGetLastError();
    launch_end(stream);
    if (err != cudaSuccess) return err;
    launch_begin(K_NORM_DWEIGHT, stream);
    err = launch_kernel(dweight_kernel, dim3((n.d_model + 31) / 32), dim3(32, kShares), 0, stream, true, part, blocks,
                        n.d_model, dweight);
    launch_end(stream);
    return err;
}

cudaError_t launch_quantize_rows(int64_t rows, int cols, int dtype, const void *x, void *q, float *scale,
                                 cudaStream_t stream) {
    if (rows == 0) return cudaSuccess;
    launch_begin(K_QUANTIZE_ROWS, stream);
    if (dtype == SWITCH_F32) quantize_typed<float>(rows, cols, x, q, scale, stream);
    else quantize_typed<__nv_bfloat16>(rows, cols, x, q, scale, stream);
    const cudaError_t err = cudaGetLastError();
    launch_end(stream);
    return err;
}

}  // namespace switchmoe
