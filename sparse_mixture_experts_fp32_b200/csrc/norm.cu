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
// there and written once.  A group of `tpr` threads holds a row, 8 elements
// (16 or 32 bytes) per thread and step; widths that are no multiple of 8 take
// the same kernels with one element per thread and step, since the rows then
// start at any alignment.  Sums and the norm are float32 (at most 32 terms per
// thread, then a tree); the maxima are taken on the bit patterns of |v|, whose
// order is that of the values and puts NaN on top, so that a row with a NaN
// gets a NaN scale.
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace switchmoe {
namespace {

constexpr float kE4m3Max = 448.f;

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
// of the block calls it.  `part` has a slot per warp of the block.
__device__ __forceinline__ float row_sum(float v, int tpr, float *part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr == 32) return v;
    const int tid = threadIdx.y * tpr + threadIdx.x, warp = tid >> 5, warps = tpr >> 5, w0 = threadIdx.y * warps;
    __syncthreads();
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
    __syncthreads();
    if ((tid & 31) == 0) p[warp] = v;
    __syncthreads();
    uint32_t s = 0;
    for (int w = 0; w < warps; ++w) s = max(s, p[w0 + w]);
    return s;
}

// The row in registers -> e4m3 and its scale.
template <int VEC, int ITERS>
__device__ __forceinline__ void quantize_row(const float (&v)[ITERS][VEC], int d, int tpr, float *part, bool live,
                                             uint8_t *q, float *scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) top = max(top, __float_as_uint(v[i][k]) & 0x7fffffffu);
    const float s = __fdiv_rn(__uint_as_float(row_max(top, tpr, part)), kE4m3Max);
    if (!live) return;
    if (threadIdx.x == 0) *scale = s;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int j = (i * tpr + (int)threadIdx.x) * VEC;
        if (j >= d) break;
        float u[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) u[k] = s == 0.f ? 0.f : __fdiv_rn(v[i][k], s);  // a row of zeros: scale 0
        store_e4m3<VEC>(q + j, u);
    }
}

template <typename R, typename D, typename O, int VEC, int ITERS>
__global__ void __launch_bounds__(ITERS * VEC == 32 ? 256 : 1024) norm_fwd_kernel(const R *residual, const D *delta, const float *__restrict__ weight, R *sum, O *out,
                                float *__restrict__ scale, float *__restrict__ rstd, int64_t T, int d, float eps) {
    __shared__ float part[32];
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
            if constexpr (!std::is_same<D, None>::value) {
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
    if constexpr (!std::is_same<D, None>::value) {
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
    const float r = __frcp_rn(__fsqrt_rn(row_sum(ss, tpr, part) / (float)d + eps));
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
        quantize_row<VEC, ITERS>(s, d, tpr, part, live, reinterpret_cast<uint8_t *>(out) + row, scale + t);
    } else {
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
            if (live && j < d) store_row<O, VEC>(out + row + j, s[i]);
        }
    }
}

template <typename R, int VEC, int ITERS>
__global__ void __launch_bounds__(1024) quantize_rows_kernel(const R *__restrict__ x, uint8_t *__restrict__ q, float *__restrict__ scale,
                                     int64_t rows, int cols) {
    __shared__ float part[32];
    const int tpr = blockDim.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < rows;
    const int64_t row = live ? t * cols : 0;
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

// Each block takes every gridDim-th group of blockDim.y rows, keeps the
// columns' sums of g * s * rstd of its rows in registers and leaves their sum
// over its rows in part_dw[block]; dweight_kernel adds the blocks in order.
template <typename R, int VEC, int ITERS>
__global__ void __launch_bounds__(ITERS * VEC == 32 ? 256 : 1024) norm_bwd_kernel(const R *__restrict__ sum, const float *__restrict__ weight,
                                const float *__restrict__ rstd, const float *dout, const float *dsum, float *dres,
                                float *__restrict__ part_dw, int64_t T, int d) {
    extern __shared__ float columns[];  // [blockDim.y][d] when a block holds several rows
    __shared__ float part[32];
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
    for (int64_t t0 = (int64_t)blockIdx.x * blockDim.y; t0 < T; t0 += step) {
        const int64_t t = t0 + threadIdx.y;
        const bool live = t < T;
        const int64_t row = live ? t * d : 0;
        float h[ITERS][VEC], g[ITERS][VEC];
        const float r = live ? rstd[t] : 0.f;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
#pragma unroll
            for (int k = 0; k < VEC; ++k) h[i][k] = g[i][k] = 0.f;
            if (live && j < d) {
                load_row<R, VEC>(sum + row + j, h[i]);
                load_row<float, VEC>(dout + row + j, g[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < ITERS; ++i)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                h[i][k] *= r;
                dw[i][k] = fmaf(g[i][k], h[i][k], dw[i][k]);
                g[i][k] *= w[i][k];
                dot = fmaf(g[i][k], h[i][k], dot);
            }
        const float m = row_sum(dot, tpr, part) / (float)d;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = (i * tpr + (int)threadIdx.x) * VEC;
            if (live && j < d) {
                float u[VEC];
#pragma unroll
                for (int k = 0; k < VEC; ++k) u[k] = 0.f;
                if (dsum != nullptr) load_row<float, VEC>(dsum + row + j, u);
#pragma unroll
                for (int k = 0; k < VEC; ++k) u[k] += r * (g[i][k] - h[i][k] * m);
                store_row<float, VEC>(dres + row + j, u);
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

// dweight_j = sum over the blocks, in order of the row groups; 32 columns x 8
// interleaved groups of blocks per block, joined in a fixed order in float64.
__global__ void dweight_kernel(const float *__restrict__ part, int blocks, int d, float *__restrict__ dweight) {
    __shared__ double acc[8][32];
    const int j = blockIdx.x * 32 + threadIdx.x;
    pdl_wait();
    double a = 0.0;
    if (j < d)
        for (int b = threadIdx.y; b < blocks; b += 8) a += (double)part[(int64_t)b * d + j];
    acc[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && j < d) {
        for (int y = 1; y < 8; ++y) a += acc[y][threadIdx.x];
        dweight[j] = (float)a;
    }
}

// Threads per row, rows per block and steps per thread for `elems` elements of VEC.
struct RowShape {
    int tpr, rows, iters;
};
RowShape row_shape(int64_t T, int d, int vec, int few, int many) {
    const int n = (d + vec - 1) / vec;
    const int iters = (T <= 1024 && n <= 1024 * few) ? few : many;
    int tpr = 32;
    while (tpr * iters < n) tpr *= 2;
    return {tpr, tpr >= 256 ? 1 : 256 / tpr, iters};
}

template <typename R, typename D, typename O>
void norm_fwd_typed(const switch_norm_dims_t &n, const void *residual, const void *delta, const float *weight,
                    void *sum, void *out, float *scale, float *rstd, cudaStream_t stream) {
    const bool wide = n.d_model % 8 == 0;
    const RowShape s = wide ? row_shape(n.T, n.d_model, 8, 1, 4) : row_shape(n.T, n.d_model, 1, 4, 32);
    const dim3 grid((unsigned)((n.T + s.rows - 1) / s.rows)), block(s.tpr, s.rows);
#define SWITCH_NORM_FWD(V, I)                                                                                  \
    norm_fwd_kernel<R, D, O, V, I><<<grid, block, 0, stream>>>(                                                \
        static_cast<const R *>(residual), static_cast<const D *>(delta), weight, static_cast<R *>(sum),        \
        static_cast<O *>(out), scale, rstd, n.T, n.d_model, n.eps)
    if (wide && s.iters == 1) SWITCH_NORM_FWD(8, 1);
    else if (wide) SWITCH_NORM_FWD(8, 4);
    else if (s.iters == 4) SWITCH_NORM_FWD(1, 4);
    else SWITCH_NORM_FWD(1, 32);
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
#define SWITCH_NORM_BWD(V, I)                                                                                  \
    norm_bwd_kernel<R, V, I><<<blocks, block, smem, stream>>>(static_cast<const R *>(sum), weight, rstd, dout, \
                                                              dsum, dres, part, n.T, n.d_model)
    if (n.d_model % 8 == 0) {
        if (s.iters == 1) SWITCH_NORM_BWD(8, 1);
        else SWITCH_NORM_BWD(8, 4);
    } else {
        if (s.iters == 4) SWITCH_NORM_BWD(1, 4);
        else SWITCH_NORM_BWD(1, 32);
    }
#undef SWITCH_NORM_BWD
}

template <typename R>
void quantize_typed(int64_t rows, int cols, const void *x, void *q, float *scale, cudaStream_t stream) {
    const bool wide = cols % 8 == 0;
    const RowShape s = wide ? row_shape(rows, cols, 8, 1, 4) : row_shape(rows, cols, 1, 4, 32);
    const dim3 grid((unsigned)((rows + s.rows - 1) / s.rows)), block(s.tpr, s.rows);
#define SWITCH_QUANT(V, I)                                                                      \
    quantize_rows_kernel<R, V, I><<<grid, block, 0, stream>>>(static_cast<const R *>(x),        \
                                                              static_cast<uint8_t *>(q), scale, rows, cols)
    if (wide && s.iters == 1) SWITCH_QUANT(8, 1);
    else if (wide) SWITCH_QUANT(8, 4);
    else if (s.iters == 4) SWITCH_QUANT(1, 4);
    else SWITCH_QUANT(1, 32);
#undef SWITCH_QUANT
}

RowShape bwd_shape(const switch_norm_dims_t &n) {
    return n.d_model % 8 == 0 ? row_shape(n.T, n.d_model, 8, 1, 4) : row_shape(n.T, n.d_model, 1, 4, 32);
}

int bwd_blocks(const switch_norm_dims_t &n) {
    const RowShape s = bwd_shape(n);
    const int64_t groups = (n.T + s.rows - 1) / s.rows;
    return (int)(groups < kNormBwdBlocks ? groups : kNormBwdBlocks);
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
    err = launch_kernel(dweight_kernel, dim3((n.d_model + 31) / 32), dim3(32, 8), 0, stream, true, part, blocks,
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
