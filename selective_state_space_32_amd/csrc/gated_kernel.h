// The gated linear recurrence, one state per channel:
//
//   log a_t = A[d] sigmoid(r_t)                      (A <= 0: the decay a_t lies in (0, 1])
//   h_t     = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(g_t) x_t
//   y_t     = h_t silu(z_t)                          (z optional)
//
// and its gradients.
#pragma once

#include <float.h>

#include "device_math.h"

namespace ssm {

// 1 - a^2 = -expm1(u), u = 2 log a <= 0, given a and y = log2(a).  Near a = 1 the difference
// loses every digit that a was rounded in, so for |u| < 1/4 the series -u (1 + u/2 + u^2/6 +
// ...) is used: its dropped terms are below u^6/5040 < 5e-8 of the value, and 1 - a^2 above
// the threshold is at least 0.22 (an ulp of a^2 costs it 4e-7).
__device__ __forceinline__ float one_minus_square(float y, float a) {
    const float u = y * (2.0f * kLn2);
    float p = fmaf(u, 1.0f / 720.0f, 1.0f / 120.0f);
    p = fmaf(p, u, 1.0f / 24.0f);
    p = fmaf(p, u, 1.0f / 6.0f);
    p = fmaf(p, u, 0.5f);
    p = -u * fmaf(p, u, 1.0f);
    return fabsf(u) < 0.25f ? p : fmaf(-a, a, 1.0f);
}

constexpr int kGatedCkpt = 16;   // tokens per stored state

// Forward, one lane per channel: the tokens in order, the state before every kGatedCkpt-th
// stored.
template <typename IO>
__global__ void __launch_bounds__(64)
gated_scan_kernel(const IO *__restrict__ x, const IO *__restrict__ r, const IO *__restrict__ g,
                  const float *__restrict__ A, const IO *__restrict__ z, const float *h0,
                  const int32_t *__restrict__ seq_lens, IO *__restrict__ y, float *last, float *__restrict__ ckpt,
                  int64_t L, int64_t D, int64_t tiles) {
    const int64_t b = blockIdx.x / tiles, d = (blockIdx.x - b * tiles) * 64 + threadIdx.x;
    if (d >= D) return;
    const int64_t Lb = seq_lens ? min((int64_t)max(seq_lens[b], 0), L) : L;
    const int64_t nck = (L + kGatedCkpt - 1) / kGatedCkpt;
    const float a2 = A[d] * kLog2e;
    float h = h0 ? h0[b * D + d] : 0.0f;
    for (int64_t t = 0; t < Lb; ++t) {
        const int64_t e = (b * L + t) * D + d;
        if (ckpt && t % kGatedCkpt == 0) ckpt[(b * nck + t / kGatedCkpt) * D + d] = h;
        const float s = sigmoid_f32(io<IO>::ld(r, e)), i = sigmoid_f32(io<IO>::ld(g, e));
        const float la = a2 * s, a = hw_exp2(la);
        const float q = one_minus_square(la, a);
        h = fmaf(a, h, __builtin_amdgcn_sqrtf(q) * i * io<IO>::ld(x, e));
        if (y) io<IO>::st(y, e, z ? h * silu_f32(io<IO>::ld(z, e)) : h);
    }
    if (y)
        for (int64_t t = Lb; t < L; ++t) io<IO>::st(y, (b * L + t) * D + d, 0.0f);
    if (last) last[b * D + d] = h;
}

// Backward, one lane per channel: tiles of kGatedCkpt tokens from the last to the first, the
// tile's states recomputed from its stored state.  dA's share of sequence b goes to part[b].
template <typename IO>
__global__ void __launch_bounds__(64)
gated_bwd_kernel(const IO *__restrict__ x, const IO *__restrict__ r, const IO *__restrict__ g,
                 const float *__restrict__ A, const IO *__restrict__ z, const int32_t *__restrict__ seq_lens,
                 const IO *__restrict__ dy, const float *__restrict__ dlast, const float *__restrict__ ckpt,
                 IO *__restrict__ dx, IO *__restrict__ dr, IO *__restrict__ dg, IO *__restrict__ dz,
                 float *__restrict__ part, float *__restrict__ dh0, int64_t L, int64_t D, int64_t tiles) {
    const int64_t b = blockIdx.x / tiles, d = (blockIdx.x - b * tiles) * 64 + threadIdx.x;
    if (d >= D) return;
    const int64_t Lb = seq_lens ? min((int64_t)max(seq_lens[b], 0), L) : L;
    const int64_t nck = (L + kGatedCkpt - 1) / kGatedCkpt;
    const float Ad = A[d], a2 = Ad * kLog2e;
    float G = dlast ? dlast[b * D + d] : 0.0f, dAd = 0.0f;
    for (int64_t j = (Lb + kGatedCkpt - 1) / kGatedCkpt - 1; j >= 0; --j) {
        const int n = (int)min((int64_t)kGatedCkpt, Lb - j * kGatedCkpt);
        float hs[kGatedCkpt + 1];
        hs[0] = ckpt[(b * nck + j) * D + d];
#pragma unroll
        for (int k = 0; k < kGatedCkpt; ++k) {
            if (k < n) {
                const int64_t e = (b * L + j * kGatedCkpt + k) * D + d;
                const float s = sigmoid_f32(io<IO>::ld(r, e)), i = sigmoid_f32(io<IO>::ld(g, e));
                const float la = a2 * s, a = hw_exp2(la);
                hs[k + 1] = fmaf(a, hs[k], __builtin_amdgcn_sqrtf(one_minus_square(la, a)) * i * io<IO>::ld(x, e));
            }
        }
#pragma unroll
        for (int k = kGatedCkpt - 1; k >= 0; --k) {
            if (k < n) {
                const int64_t e = (b * L + j * kGatedCkpt + k) * D + d;
                const float s = sigmoid_f32(io<IO>::ld(r, e)), i = sigmoid_f32(io<IO>::ld(g, e));
                const float xx = io<IO>::ld(x, e);
                const float la = a2 * s, a = hw_exp2(la);
                const float q = one_minus_square(la, a);
                const float rb = fabsf(q) < FLT_MIN ? 0.0f : __builtin_amdgcn_rsqf(q), beta = q * rb;
                float dh = io<IO>::ld(dy, e);
                if (z) {
                    const float zz = io<IO>::ld(z, e), sz = sigmoid_f32(zz);
                    io<IO>::st(dz, e, dh * hs[k + 1] * (sz * fmaf(zz, 1.0f - sz, 1.0f)));
                    dh *= zz * sz;
                }
                const float lam = dh + G;
                G = a * lam;
                const float lb = lam * beta * i;
                io<IO>::st(dx, e, lb);
                io<IO>::st(dg, e, lb * xx * (1.0f - i));
                const float dla = fmaf(G, hs[k], -lam * (i * xx) * (a * a * rb));
                io<IO>::st(dr, e, dla * Ad * (s * (1.0f - s)));
                dAd = fmaf(dla, s, dAd);
            }
        }
    }
    for (int64_t t = Lb; t < L; ++t) {
        const int64_t e = (b * L + t) * D + d;
        io<IO>::st(dx, e, 0.0f);
        io<IO>::st(dr, e, 0.0f);
        io<IO>::st(dg, e, 0.0f);
        if (z) io<IO>::st(dz, e, 0.0f);
    }
    part[b * D + d] = dAd;
    if (dh0) dh0[b * D + d] = G;
}

// dA[d] = sum of the n rows of part, in order.
static __global__ void __launch_bounds__(256)
column_sum_kernel(const float *__restrict__ part, float *__restrict__ out, int64_t n, int64_t D) {
    const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (d >= D) return;
    float s = 0.0f;
    for (int64_t k = 0; k < n; ++k) s += part[k * D + d];
    out[d] = s;
}

// One token of every sequence, the state updated in place.
template <typename IO>
__global__ void __launch_bounds__(256)
gated_step_kernel(float *__restrict__ state, const IO *__restrict__ x, const IO *__restrict__ r,
                  const IO *__restrict__ g, const float *__restrict__ A, const IO *__restrict__ z,
                  IO *__restrict__ y, int64_t n, int64_t D) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= n) return;
    const float s = sigmoid_f32(io<IO>::ld(r, e)), i = sigmoid_f32(io<IO>::ld(g, e));
    const float la = A[e % D] * kLog2e * s, a = hw_exp2(la);
    const float h = fmaf(a, state[e], __builtin_amdgcn_sqrtf(one_minus_square(la, a)) * i * io<IO>::ld(x, e));
    state[e] = h;
    io<IO>::st(y, e, z ? h * silu_f32(io<IO>::ld(z, e)) : h);
}

}  // namespace ssm
