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
// or 32 bytes) per thread.  The eights are those of the whole tensor, which
// start on 16 bytes whatever the width is; where the width is no multiple of 8
// (ODD) a row's first and last eight are read and written one by one.  Blocks
// live for one row group (a loop over rows that loads the next one early
// measured 20 % slower: 237 us); only the gradient, which keeps column sums,
// loops.  Sums and the norm are float32 (8 terms per thread, then a tree); the
// maxima are taken on the bit patterns of |v|, whose order is that of the values
// and puts NaN on top, so that a row with a NaN gets a NaN scale.
//
// Measured on B200s (copy bandwidth 6549 GB/s): 131072 x 1024 bfloat16 +
// float32 -> bfloat16 193 us (7.0 TB/s), its gradient 304-312 us (6.0-6.2 TB/s);
// 8192 x 768 float32 + float32 -> 8 bits 16.2 us (5.0 TB/s); 131072 x 1024
// bfloat16 to 8 bits 81-84 us (4.8-5.0 TB/s).  At widths that are no multiple of
// 8 (1001) 152 us for 65536 rows to bfloat16 (4.3 TB/s), 113 us from bfloat16 to
// 8 bits (1.7 TB/s): a row's ends go one by one, in a form of 71 registers.
#include <cuda_fp8.h>

#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace switchmoe {
namespace {

constexpr float kE4m3Max = 448.f;
struct None {};  // no delta

// Eight elements of a row of d, from element j on.  ODD: j may be up to 7
// before the row, and the eight may reach past its end; what is not of the row
// is neither read (0 instead) nor written.  `ones`: every eight one by one.
template <typename T, bool ODD>
__device__ __forceinline__ void load8(const T *row, int j, int d, bool ones, float (&v)[8]) {
    const T *p = row + j;
    if (ODD && (ones || j < 0 || j + 8 > d)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = j + k >= 0 && j + k < d ? Elem<T>::load(p, k) : 0.f;
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

// The same of a vector that starts on 16 bytes, whatever j is: ODD reads it one by one (it stays in L1).
template <bool ODD>
__device__ __forceinline__ void load_weight(const float *w, int j, int d, float (&v)[8]) {
    if constexpr (ODD) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = j + k >= 0 && j + k < d ? __ldg(w + j + k) : 0.f;
    } else {
        load8<float, false>(w, j, d, false, v);
    }
}

template <typename T, bool ODD>
__device__ __forceinline__ void store8(T *row, int j, int d, bool ones, const float (&v)[8]) {
    T *p = row + j;
    if (ODD && (ones || j < 0 || j + 8 > d)) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (j + k >= 0 && j + k < d) Elem<T>::store(p, k, v[k]);
    } else if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
}

template <bool ODD>
__device__ __forceinline__ void store8_e4m3(uint8_t *row, int j, int d, bool ones, const float (&v)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi =
            __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    if (ODD && (ones || j < 0 || j + 8 > d)) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (j + k >= 0 && j + k < d) row[j + k] = (uint8_t)(w[k / 4] >> (8 * (k % 4)));
    } else {
        *reinterpret_cast<uint2 *>(row + j) = make_uint2(w[0], w[1]);
    }
}

// First element of step i of this thread in row t: eights of the whole tensor,
// so that they start on 16 bytes (8 in 8 bits) in every row.
template <bool ODD>
__device__ __forceinline__ int first_of(int i, int64_t t, int d, bool ones) {
    return (i * (int)blockDim.x + (int)threadIdx.x) * 8 - (ODD && !ones ? (int)((t * d) & 7) : 0);
}

// Whether a block's threads, at 1024 of them, are too few for a row's eights
// and hold the row from its own beginning instead (the last widths below 8192
// and, in four steps, below 32768).
template <bool ODD>
__device__ __forceinline__ bool by_ones(int steps, int d) {
    return ODD && (int)blockDim.x * steps * 8 < d + 7;
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

// Scale of a row whose largest |v| has the bits `top`, and the rounding of its
// values.  e4m3's rounding of v / s is that of t = v * (1 / s), which is within
// 2 units in the last place of the quotient, unless t is as close to the middle
// between two e4m3 values: in the normal range those have the 20 low bits
// 0x80000.  Eights with such a t, or with one below the normal range (2^-6), are
// divided.  (131072 x 1024 bfloat16 took 116 us in the first kernel, which divided
// every element; with this and its other steps 81 us.)
struct Quantizer {
    float s, inv;
    bool tiny;  // 1 / s may overflow
    __device__ explicit Quantizer(uint32_t top) {
        s = __fdiv_rn(__uint_as_float(top), kE4m3Max);
        inv = __frcp_rn(s);
        tiny = s < 1e-30f;
    }
    __device__ __forceinline__ bool below_normal(float least) const { return least * inv < 0.0157f; }
    // `divide`: an element may be below the normal range.  SEEK: look for one (a zero counts).
    template <bool ODD, bool SEEK>
    __device__ __forceinline__ void store(uint8_t *q, int j, int d, bool ones, const float (&v)[8], bool divide) const {
        float u[8], least = 1.f;
        uint32_t middle = 0xffffffffu;  // least distance from 8 below a middle
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            u[k] = v[k] * inv;
            middle = __viaddmin_u32(__float_as_uint(u[k]) & 0xfffffu, 0u - 0x7fff8u, middle);
            if (SEEK) least = fminf(least, ODD && u[k] == 0.f ? 1.f : fabsf(u[k]));  // (ODD: zeros beside the row)
        }
        if (tiny || divide || middle <= 0x10u || (SEEK && least < 0.015625f)) {
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = s == 0.f ? 0.f : __fdiv_rn(v[k], s);  // a row of zeros: scale 0
        }
        store8_e4m3<ODD>(q, j, d, ones, u);
    }
};

// Whether the mean of a row's squares (with eps) is beyond float32's range
// (values from about 1e19 up), or so small that squares may have lost bits (below
// about 1e-15): the row is then scaled by a power of two and summed once more.
__device__ __forceinline__ bool beyond_squares(float mean) {
    constexpr uint32_t least = 27u << 23;  // 2^-100; a NaN's bits are above an infinity's
    return __float_as_uint(mean) - least >= (255u << 23) - least;
}

template <typename R, typename D, typename O, bool ODD>
__global__ void __launch_bounds__(1024)
    norm_fwd_kernel(const R *residual, const D *delta, const float *__restrict__ weight, R *sum, O *out,
                    float *__restrict__ scale, float *__restrict__ rstd, int64_t T, int d, float eps) {
    constexpr bool kDelta = !std::is_same<D, None>::value;
    __shared__ float part[3][32];
    const int tpr = blockDim.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < T;
    const int64_t row = live ? t * d : 0;
    const bool ones = by_ones<ODD>(1, d);
    const int j = first_of<ODD>(0, t, d, ones);
    const bool mine = live && j < d;
    float s[8];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = 0.f;
    if (mine) {
        load8<R, ODD>(residual + row, j, d, ones, s);
        if constexpr (kDelta) {
            float a[8];
            load8<D, ODD>(delta + row, j, d, ones, a);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[k] += a[k];
                // the sum is normalised as it is stored: the backward pass reads the stored one
                if constexpr (sizeof(R) == 2) s[k] = bf16_bits_to_float(float_to_bf16_bits(s[k]));
            }
            if (sum != nullptr) store8<R, ODD>(sum + row, j, d, ones, s);
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(s[k], s[k], ss);
    const float mean = row_sum(ss, tpr, part[0]) / (float)d + eps;
    float r = __frcp_rn(__fsqrt_rn(mean)), r_stored = r;
    if (__builtin_expect(beyond_squares(mean), 0)) {  // (the same in all threads that share a row or a barrier)
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(s[k]) & 0x7fffffffu);
        top = row_max(top, tpr, part[2]);
        if (top < 0x7f800000u) {  // (a row with a NaN or an infinity stays as it is)
            const float m = fmaxf(__uint_as_float(top), __fsqrt_rn(eps));
            const int down = m > 0.f ? -ilogbf(m) : 0;
            const float a = scalbnf(1.f, down / 2), b = scalbnf(1.f, down - down / 2);
            ss = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = s[k] * a * b, ss = fmaf(s[k], s[k], ss);
            r = __frcp_rn(__fsqrt_rn(row_sum(ss, tpr, part[0]) / (float)d + eps * a * b * a * b));
            r_stored = r * a * b;
            if (m == 0.f) r = 0.f;  // zeros without an eps: 0 beside an infinite rstd
        }
    }
    if (live && threadIdx.x == 0 && rstd != nullptr) rstd[t] = r_stored;
    if (j < d) {
        float w[8];
        load_weight<ODD>(weight, j, d, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] = s[k] * r * w[k];
    }
    if constexpr (sizeof(O) == 1) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(s[k]) & 0x7fffffffu);
        const Quantizer z(row_max(top, tpr, part[1]));
        if (live && threadIdx.x == 0) scale[t] = z.s;
        if (mine) z.store<ODD, true>(reinterpret_cast<uint8_t *>(out) + row, j, d, ones, s, false);
    } else {
        if (mine) store8<O, ODD>(out + row, j, d, ones, s);
    }
}

template <typename R, int ITERS, int THREADS, bool ODD>
__global__ void __launch_bounds__(THREADS, THREADS == 256 && sizeof(R) == 2 && !ODD ? 6 : 1)
    quantize_rows_kernel(const R *__restrict__ x, uint8_t *__restrict__ q, float *__restrict__ scale, int64_t rows,
                         int cols) {
    __shared__ float part[32];
    const int tpr = blockDim.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < rows;
    const int64_t row = live ? t * cols : 0;
    if constexpr (!ODD && sizeof(R) == 2) {
        // the row stays in its 16 bits until it is rounded: half the registers, twice the rows in flight
        uint4 raw[ITERS];
        uint32_t top2 = 0, low2 = 0xffffffffu;  // of |x|, two at a time; low2 is one less, so that zeros do not count
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = first_of<false>(i, t, cols, false);
            raw[i] = live && j < cols ? *reinterpret_cast<const uint4 *>(x + row + j) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a = w[k] & 0x7fff7fffu;
                top2 = __vmaxu2(top2, a);
                low2 = __viaddmin_u16x2(a, 0xffffffffu, low2);
            }
        }
        const Quantizer z(row_max(max(top2 << 16, top2 & 0xffff0000u), tpr, part));
        if (!live) return;
        if (threadIdx.x == 0) scale[t] = z.s;
        const uint32_t low = min(low2 & 0xffffu, low2 >> 16);
        const bool small = low < 0x7f80u && z.below_normal(bf16_bits_to_float((uint16_t)(low + 1)));
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = first_of<false>(i, t, cols, false);
            if (j >= cols) break;
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            float v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            z.store<false, false>(q + row, j, cols, false, v, small);
        }
    } else {
        const bool ones = by_ones<ODD>(ITERS, cols);
        float v[ITERS][8];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = first_of<ODD>(i, t, cols, ones);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
            if (live && j < cols) load8<R, ODD>(x + row, j, cols, ones, v[i]);
        }
#pragma unroll
        for (int i = 0; i < ITERS; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[i][k]) & 0x7fffffffu);
        const Quantizer z(row_max(top, tpr, part));
        if (!live) return;
        if (threadIdx.x == 0) scale[t] = z.s;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int j = first_of<ODD>(i, t, cols, ones);
            if (j < cols) z.store<ODD, true>(q + row, j, cols, ones, v[i], false);
        }
    }
}

// Each block takes every gridDim-th group of blockDim.y rows, keeps the
// columns' sums of g * s * rstd of its rows in registers and leaves their sum
// over its rows in part_dw[block]; dweight_kernel adds the blocks in order.
// A thread holds 8 elements of a row, so that enough blocks fit on an SM to
// keep memory busy (32 elements: 600 us at 131072 x 1024, 8: 304 us), and loads
// the next row's while this one's sum is formed.  Its columns are the same in
// all its rows: ODD takes a number of blocks that makes them 8 rows apart.
template <typename R, int THREADS, bool ODD>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? (ODD ? 3 : 4) : 1)
    norm_bwd_kernel(const R *__restrict__ sum, const float *__restrict__ weight, const float *__restrict__ rstd,
                    const float *dout, const float *dsum, float *dres, float *__restrict__ part_dw, int64_t T, int d) {
    extern __shared__ float columns[];  // [blockDim.y][d] when a block holds several rows
    __shared__ float part[2][32];
    const int tpr = blockDim.x;
    const int64_t t_first = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool ones = by_ones<ODD>(1, d);
    const int j = first_of<ODD>(0, t_first, d, ones);
    float w[8], dw[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = dw[k] = 0.f;
    if (j < d) load_weight<ODD>(weight, j, d, w);
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    float h[8], g[8];
    float r = 0.f;
    auto load = [&](int64_t t) {
        const bool live = t < T;
        r = live ? rstd[t] : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = g[k] = 0.f;
        if (live && j < d) {
            load8<R, ODD>(sum + t * d, j, d, ones, h);
            load8<float, ODD>(dout + t * d, j, d, ones, g);
        }
    };
    load(t_first);
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * blockDim.y; t0 < T; t0 += step) {
        const int64_t t = t0 + threadIdx.y;
        const bool mine = t < T && j < d;
        const float rt = r;
        float u[8], b[8];
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = 0.f;
        if (mine && dsum != nullptr) load8<float, ODD>(dsum + t * d, j, d, ones, u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float hat = h[k] * rt;
            dw[k] = fmaf(g[k], hat, dw[k]);
            const float gw = g[k] * w[k];
            dot = fmaf(gw, hat, dot);
            u[k] = fmaf(rt, gw, u[k]);
            b[k] = rt * hat;
        }
        load(t + step);
        const float m = row_sum(dot, tpr, part[turn]) / (float)d;
        turn ^= 1;
        if (mine) {
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = fmaf(-m, b[k], u[k]);
            store8<float, ODD>(dres + t * d, j, d, ones, u);
        }
    }
    float *to = blockDim.y == 1 ? part_dw + (int64_t)blockIdx.x * d : columns + threadIdx.y * d;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (j + k >= 0 && j + k < d) to[j + k] = dw[k];
    if (blockDim.y > 1) {
        __syncthreads();
        const int threads = blockDim.x * blockDim.y;
        for (int c = threadIdx.y * tpr + threadIdx.x; c < d; c += threads) {
            float a = 0.f;
            for (int y = 0; y < (int)blockDim.y; ++y) a += columns[y * d + c];
            part_dw[(int64_t)blockIdx.x * d + c] = a;
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
    const int tpr = n > 1024 * iters ? 1024 : (n + 32 * iters - 1) / (32 * iters) * 32;
    return {tpr, tpr == 32 ? 8 : tpr >= 128 ? 1 : 128 / tpr, iters};
}

// Eights that cover a row of d elements, wherever in one it begins.
int eights(int d) { return d % 8 == 0 ? d / 8 : (d + 7 + 7) / 8; }

template <typename R, typename D, typename O>
void norm_fwd_typed(const switch_norm_dims_t &n, const void *residual, const void *delta, const float *weight,
                    void *sum, void *out, float *scale, float *rstd, cudaStream_t stream) {
    RowShape s = shape_of(eights(n.d_model), 1);
    if (s.tpr > 32) s.rows = 1;  // (rows that share a barrier would have to agree on a second sum)
    const dim3 grid((unsigned)((n.T + s.rows - 1) / s.rows)), block(s.tpr, s.rows);
    auto *kernel = n.d_model % 8 == 0 ? norm_fwd_kernel<R, D, O, false> : norm_fwd_kernel<R, D, O, true>;
    kernel<<<grid, block, 0, stream>>>(static_cast<const R *>(residual), static_cast<const D *>(delta), weight,
                                       static_cast<R *>(sum), static_cast<O *>(out), scale, rstd, n.T, n.d_model,
                                       n.eps);
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
    const bool odd = n.d_model % 8 != 0;
    auto *kernel = s.tpr <= 256 ? (odd ? norm_bwd_kernel<R, 256, true> : norm_bwd_kernel<R, 256, false>)
                                : (odd ? norm_bwd_kernel<R, 1024, true> : norm_bwd_kernel<R, 1024, false>);
    kernel<<<blocks, block, smem, stream>>>(static_cast<const R *>(sum), weight, rstd, dout, dsum, dres, part, n.T,
                                            n.d_model);
}

template <typename R>
void quantize_typed(int64_t rows, int cols, const void *x, void *q, float *scale, cudaStream_t stream) {
    // Four steps per thread, a row to a warp, once there are rows enough to fill the GPU with warps: 16384 x 1024
    // takes 15 us so and 19 us with one step, 4096 x 1024 6.2 us and 5.8 us.
    const bool large = rows * (int64_t)cols > (1 << 23) || cols > 8192, odd = cols % 8 != 0;
    const RowShape s = shape_of(eights(cols), large ? 4 : 1);
    const dim3 grid((unsigned)((rows + s.rows - 1) / s.rows)), block(s.tpr, s.rows);
    auto *kernel =
        s.iters == 1 ? (odd ? quantize_rows_kernel<R, 1, 1024, true> : quantize_rows_kernel<R, 1, 1024, false>)
        : s.tpr <= 256 ? (odd ? quantize_rows_kernel<R, 4, 256, true> : quantize_rows_kernel<R, 4, 256, false>)
                       : (odd ? quantize_rows_kernel<R, 4, 1024, true> : quantize_rows_kernel<R, 4, 1024, false>);
    kernel<<<grid, block, 0, stream>>>(static_cast<const R *>(x), static_cast<uint8_t *>(q), scale, rows, cols);
}

RowShape bwd_shape(const switch_norm_dims_t &n) { return shape_of(eights(n.d_model), 1); }

int bwd_blocks(const switch_norm_dims_t &n) {
    const RowShape s = bwd_shape(n);
    const int64_t groups = (n.T + s.rows - 1) / s.rows;
    // As many blocks as are resident: 64 registers a thread leave an SM 1024 threads (80, for odd widths, 768).
    const bool odd = n.d_model % 8 != 0;
    const int64_t most = (int64_t)kNormBwdSms * (odd && s.tpr <= 256 ? 768 : 1024) / (s.tpr * s.rows);
    const int64_t blocks = groups < most ? groups : most;
    return (int)(odd ? (blocks + 7) / 8 * 8 : blocks);
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
