// Layer norm over the last axis, with the residual sum in front of it, and its gradients:
//
//   s = x + residual (rounded to the type it is kept in),  mu = mean(s),
//   rstd = 1 / sqrt(mean((s - mu)^2) + eps),  y = (s - mu) rstd w + b
//   ds = rstd (dy w - mean(dy w) - xh mean(dy w xh)) + dresidual,  xh = (s - mu) rstd
//   dw = sum over rows of dy xh,  db = sum over rows of dy
#pragma once

#include "device_math.h"

namespace ssm {

constexpr int kNormThreads = 256;

// Sum over the workgroup, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) v += __shfl_xor(v, k);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int k = 1; k < kNormThreads / 64; ++k) s += red[k];
    return s;
}

// One workgroup per row, three passes over it.  S: the type of residual and sum.
template <typename IO, typename S>
__global__ void __launch_bounds__(kNormThreads)
layernorm_fwd_kernel(const IO *__restrict__ x, const S *res, const float *__restrict__ w,
                     const float *__restrict__ bias, float eps, IO *__restrict__ y, S *sum,
                     float *__restrict__ mean, float *__restrict__ rstd, int64_t D) {
    __shared__ float red[kNormThreads / 64];
    const int64_t row = blockIdx.x, o = row * D;
    auto value = [&](int64_t k) {
        float v = io<IO>::ld(x, o + k);
        if (res) v += io<S>::ld(res, o + k);
        if constexpr (sizeof(S) == 2) v = bf16_to_f32(f32_to_bf16(v));
        return v;
    };
    float m = 0.0f;
    for (int64_t k = threadIdx.x; k < D; k += kNormThreads) m += value(k);
    m = block_sum(m, red) / (float)D;
    float q = 0.0f;
    for (int64_t k = threadIdx.x; k < D; k += kNormThreads) {
        const float c = value(k) - m;
        q = fmaf(c, c, q);
    }
    const float rs = 1.0f / sqrtf(block_sum(q, red) / (float)D + eps);
    for (int64_t k = threadIdx.x; k < D; k += kNormThreads) {
        const float v = value(k), n = (v - m) * rs;
        if (sum) io<S>::st(sum, o + k, v);
        io<IO>::st(y, o + k, bias ? fmaf(n, w[k], bias[k]) : n * w[k]);
    }
    if (threadIdx.x == 0) {
        if (mean) mean[row] = m;
        if (rstd) rstd[row] = rs;
    }
}

template <typename IO, typename S>
__global__ void __launch_bounds__(kNormThreads)
layernorm_bwd_kernel(const IO *__restrict__ dy, const S *__restrict__ s, const float *__restrict__ w,
                     const float *__restrict__ mean, const float *__restrict__ rstd, const S *dres, S *ds,
                     IO *__restrict__ dx, int64_t D) {
    __shared__ float red[kNormThreads / 64];
    const int64_t row = blockIdx.x, o = row * D;
    const float m = mean[row], rs = rstd[row];
    float p = 0.0f, q = 0.0f;
    for (int64_t k = threadIdx.x; k < D; k += kNormThreads) {
        const float t = io<IO>::ld(dy, o + k) * w[k];
        p += t;
        q = fmaf(t, (io<S>::ld(s, o + k) - m) * rs, q);
    }
    p = block_sum(p, red) / (float)D;
    q = block_sum(q, red) / (float)D;
    for (int64_t k = threadIdx.x; k < D; k += kNormThreads) {
        const float xh = (io<S>::ld(s, o + k) - m) * rs;
        float v = (io<IO>::ld(dy, o + k) * w[k] - p - xh * q) * rs;
        if (dres) v += io<S>::ld(dres, o + k);
        io<S>::st(ds, o + k, v);
        if (dx) io<IO>::st(dx, o + k, v);
    }
}

// The parameters' gradients over rows [blockIdx.y * rows_per, ...), one column per thread.
template <typename IO, typename S>
__global__ void __launch_bounds__(256)
layernorm_wgrad_kernel(const IO *__restrict__ dy, const S *__restrict__ s, const float *__restrict__ mean,
                       const float *__restrict__ rstd, float *__restrict__ pw, float *__restrict__ pb, int64_t M,
                       int64_t D, int64_t rows_per) {
    const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (d >= D) return;
    const int64_t r1 = min(M, (blockIdx.y + 1) * rows_per);
    float a = 0.0f, b = 0.0f;
    for (int64_t i = blockIdx.y * rows_per; i < r1; ++i) {
        const float g = io<IO>::ld(dy, i * D + d);
        a = fmaf(g, (io<S>::ld(s, i * D + d) - mean[i]) * rstd[i], a);
        b += g;
    }
    pw[blockIdx.y * D + d] = a;
    pb[blockIdx.y * D + d] = b;
}

// out[d] = sum of the n rows of part, in order (both arrays in one launch).
static __global__ void __launch_bounds__(256)
layernorm_wgrad_sum_kernel(const float *__restrict__ pw, const float *__restrict__ pb, float *__restrict__ dw,
                           float *__restrict__ db, int64_t n, int64_t D) {
    const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (d >= D) return;
    float a = 0.0f, b = 0.0f;
    for (int64_t k = 0; k < n; ++k) {
        a += pw[k * D + d];
        b += pb[k * D + d];
    }
    if (dw) dw[d] = a;
    if (db) db[d] = b;
}

}  // namespace ssm
