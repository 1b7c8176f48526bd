// Layer norm over the last axis, with the residual sum in front of it, and its gradients:
//
//   s = x + residual (rounded to the type it is kept in),  mu = mean(s),
//   rstd = 1 / sqrt(mean((s - mu)^2) + eps),  y = (s - mu) rstd w + b
//   ds = rstd (dy w - mean(dy w) - n mean(dy w n)) + dresidual,  n = (s - mu) rstd
//   dw = sum over rows of dy n,  db = sum over rows of dy
//
// Bound: HBM (every row is read once and written once).  A row is held in the registers of TPR
// threads (a wave for narrow rows, a workgroup for wide ones), NV vectors of kNormVec values each,
// so that the variance is taken from centred values without a second pass over memory.  A thread
// keeps its columns over all the rows that its workgroup takes: the weights stay in registers, and
// so do the sums over rows behind dw and db.  The next row is requested before the current one is
// reduced.  Rows wider than the registers hold take the kernels at the end, which pass over a row
// several times (its later passes come from the cache).  Measured (a copy of 1 GiB reaches 5.1 TB/s on
// this card): 16384x5120 bf16 with an fp32 residual 177 us for 1,007 MB, its backward 225 us for
// 1,342 MB; 4096x1536 fp32 backward 20 us for 76 MB; 256x5120 bf16 5.8 us for 16 MB, the latency of a
// load, two sums over a workgroup and a store.
#pragma once

#include "device_math.h"

namespace ssm {

constexpr int kNormVec = 4;   // values per access

// Sum over the wave's lanes, in every lane (row shifts, then the two row broadcasts).
__device__ __forceinline__ float wave_sum(float v) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x111, 0xf, 0xf, false));  // row_shr:1
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x112, 0xf, 0xf, false));  // row_shr:2
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x114, 0xf, 0xf, false));  // row_shr:4
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x118, 0xf, 0xf, false));  // row_shr:8
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xa, 0xf, false));  // row_bcast:15
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xc, 0xf, false));  // row_bcast:31
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sums of two values over the TPR threads of a row, in every thread.  red: the row's LDS slots, one
// pair per wave; the caller alternates between two sets, so that one barrier per sum is enough.
template <int TPR>
__device__ __forceinline__ void row_sum2(float &p, float &q, float (*red)[2]) {
    p = wave_sum(p);
    q = wave_sum(q);
    if constexpr (TPR > 64) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            red[w][0] = p;
            red[w][1] = q;
        }
        __syncthreads();
        p = red[0][0];
        q = red[0][1];
#pragma unroll
        for (int k = 1; k < TPR / 64; ++k) {
            p += red[k][0];
            q += red[k][1];
        }
    }
}
template <int TPR>
__device__ __forceinline__ float row_sum(float p, float *red) {
    p = wave_sum(p);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = p;
        __syncthreads();
        p = red[0];
#pragma unroll
        for (int k = 1; k < TPR / 64; ++k) p += red[k];
    }
    return p;
}

// kNormVec values of a row from column c on, as raw words; nothing is assumed about alignment
// beyond the element's own (rows of an odd width start anywhere).  The vector that crosses the
// row's end is read by elements, columns past it are zero.  NT: past the caches, as data that is used
// once; not where rows start inside a line, whose other part the neighbouring access wants (32768x771
// bf16 with fp32 sums: 63 us through the caches, 65 past them, backward 86 and 103; at 768 columns 54 and 52,
// 76 and 71).
template <typename T, bool NT> struct norm_vec {
    static constexpr int W = kNormVec * (int)sizeof(T) / 4;
    typedef uint32_t any_u32 __attribute__((ext_vector_type(W), aligned(sizeof(T))));
    uint32_t w[W];
    __device__ __forceinline__ void load(const T *row, int64_t c, int64_t D) {
        if (c + kNormVec <= D) {
            any_u32 v;
            if constexpr (NT) v = __builtin_nontemporal_load(reinterpret_cast<const any_u32 *>(row + c));
            else v = *reinterpret_cast<const any_u32 *>(row + c);
            __builtin_memcpy(w, &v, sizeof w);
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k] = 0;
#pragma unroll
            for (int k = 0; k < kNormVec; ++k)
                if (c + k < D) {
                    if constexpr (sizeof(T) == 2) w[k >> 1] |= (uint32_t)row[c + k] << (16 * (k & 1));
                    else w[k] = __float_as_uint(row[c + k]);
                }
        }
    }
    __device__ __forceinline__ float get(int k) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[k]);
        else return __uint_as_float((k & 1) ? (w[k >> 1] & 0xffff0000u) : (w[k >> 1] << 16));
    }
    __device__ __forceinline__ static void store(T *row, int64_t c, int64_t D, const float (&y)[kNormVec]) {
        if (c + kNormVec <= D) {
            uint32_t o[W];
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int k = 0; k < W; ++k) o[k] = f32x2_to_bf16x2(y[2 * k], y[2 * k + 1]);
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k) o[k] = __float_as_uint(y[k]);
            }
            any_u32 v;
            __builtin_memcpy(&v, o, sizeof o);
            if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<any_u32 *>(row + c));
            else *reinterpret_cast<any_u32 *>(row + c) = v;
        } else {
#pragma unroll
            for (int k = 0; k < kNormVec; ++k)
                if (c + k < D) io<T>::st(row, c + k, y[k]);
        }
    }
};

// fp32 parameters of the thread's columns (zero without the array or past the row).
__device__ __forceinline__ void load_params(const float *p, int64_t c, int64_t D, float (&o)[kNormVec]) {
    typedef float any_f32 __attribute__((ext_vector_type(kNormVec), aligned(sizeof(float))));
    if (p && c + kNormVec <= D) {
        const any_f32 v = *reinterpret_cast<const any_f32 *>(p + c);
#pragma unroll
        for (int k = 0; k < kNormVec; ++k) o[k] = v[k];
    } else {
#pragma unroll
        for (int k = 0; k < kNormVec; ++k) o[k] = p && c + k < D ? p[c + k] : 0.0f;
    }
}

// 1 / sqrt(variance + eps) of values centred with a mean that still lacks e: q / D - e^2, which is not
// below zero but for rounding (and infinite or NaN as q is).
__device__ __forceinline__ float rstd_of(float q, float inv_d, float e, float eps) {
    float var = q * inv_d;
    if (var < __builtin_inff()) var = fmaxf(fmaf(-e, e, var), 0.0f);
    return 1.0f / sqrtf(var + eps);
}

// The mean m of a first sum is off by the sum's roundings and by that of 1 / D: an ulp or several, which
// rstd makes visible where a row varies little (rows of 1900 at D = 500: 3.9e-2 of y with the default eps).
// v - m is exact there, so its mean e, summed along with the squares, is what m lacks.
// SLOTS = threads / TPR rows at a time.  S: the type of residual and sum.
template <typename IO, typename S, int TPR, int NV, bool NT>
__global__ void __launch_bounds__(TPR > 64 ? TPR : 256)
layernorm_fwd_kernel(const IO *__restrict__ x, const S *res, const float *__restrict__ w,
                     const float *__restrict__ bias, float eps, IO *__restrict__ y, S *sum,
                     float *__restrict__ mean, float *__restrict__ rstd, int64_t M, int64_t D) {
    constexpr int SLOTS = TPR > 64 ? 1 : 256 / TPR;
    __shared__ float red[TPR / 64], red2[TPR / 64][2];
    const int tid = threadIdx.x % TPR;
    const float inv_d = 1.0f / (float)D;
    float wv[NV][kNormVec], bv[NV][kNormVec];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)(j * TPR + tid) * kNormVec;
        load_params(w, c, D, wv[j]);
        load_params(bias, c, D, bv[j]);
    }
    norm_vec<IO, NT> rx[NV];
    norm_vec<S, NT> rr[NV];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPR + tid) * kNormVec;
            rx[j].load(x + row * D, c, D);
            if (res) rr[j].load(res + row * D, c, D);
        }
    };
    const int64_t step = (int64_t)gridDim.x * SLOTS;
    int64_t row = (int64_t)blockIdx.x * SLOTS + (SLOTS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0);
    if (row < M) fetch(row);
    for (; row < M; row += step) {
        float v[NV][kNormVec], m = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                float t = rx[j].get(k);
                if (res) t += rr[j].get(k);
                if constexpr (sizeof(S) == 2) t = bf16_to_f32(f32_to_bf16(t));
                v[j][k] = t;
                m += t;
            }
        if (row + step < M) fetch(row + step);
        m = row_sum<TPR>(m, red) * inv_d;
        float e = 0.0f, q = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPR + tid) * kNormVec;
            if (sum && c < D) norm_vec<S, NT>::store(sum + row * D, c, D, v[j]);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                v[j][k] = c + k < D ? v[j][k] - m : 0.0f;
                e += v[j][k];
                q = fmaf(v[j][k], v[j][k], q);
            }
        }
        row_sum2<TPR>(e, q, red2);
        e *= inv_d;
        const float rs = rstd_of(q, inv_d, e, eps), shift = -e * rs;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPR + tid) * kNormVec;
            float o[kNormVec];
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) o[k] = fmaf(fmaf(v[j][k], rs, shift), wv[j][k], bv[j][k]);
            if (c < D) norm_vec<IO, NT>::store(y + row * D, c, D, o);
        }
        if (tid == 0) {
            if (mean) mean[row] = m + e;
            if (rstd) rstd[row] = rs;
        }
    }
}

// The gradients; the sums over this workgroup's rows go to row blockIdx.x of pw and pb (if given).
template <typename IO, typename S, int TPR, int NV, bool NT>
__global__ void __launch_bounds__(TPR > 64 ? TPR : 256)
layernorm_bwd_kernel(const IO *__restrict__ dy, const S *__restrict__ s, const float *__restrict__ w,
                     const float *__restrict__ mean, const float *__restrict__ rstd, const S *dres, S *ds,
                     IO *__restrict__ dx, float *__restrict__ pw, float *__restrict__ pb, int64_t M, int64_t D) {
    constexpr int SLOTS = TPR > 64 ? 1 : 256 / TPR;
    __shared__ float red[2][TPR / 64][2];
    const int tid = threadIdx.x % TPR;
    const int slot = SLOTS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0;
    float wv[NV][kNormVec], aw[NV][kNormVec], ab[NV][kNormVec];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        load_params(w, (int64_t)(j * TPR + tid) * kNormVec, D, wv[j]);
#pragma unroll
        for (int k = 0; k < kNormVec; ++k) aw[j][k] = ab[j][k] = 0.0f;
    }
    norm_vec<IO, NT> rg[NV];
    norm_vec<S, NT> rs[NV], rd[NV];
    float m = 0.0f, r = 0.0f;
    auto fetch = [&](int64_t row) {
        m = mean[row];
        r = rstd[row];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPR + tid) * kNormVec;
            rg[j].load(dy + row * D, c, D);
            rs[j].load(s + row * D, c, D);
            if (dres) rd[j].load(dres + row * D, c, D);
        }
    };
    const int64_t step = (int64_t)gridDim.x * SLOTS;
    int64_t row = (int64_t)blockIdx.x * SLOTS + slot;
    int turn = 0;
    if (row < M) fetch(row);
    for (; row < M; row += step, turn ^= 1) {
        float t[NV][kNormVec], n[NV][kNormVec], p = 0.0f, q = 0.0f;
        norm_vec<S, NT> cd[NV];
        const float rc = r;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPR + tid) * kNormVec;
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                const float g = rg[j].get(k);
                n[j][k] = c + k < D ? (rs[j].get(k) - m) * r : 0.0f;
                aw[j][k] = fmaf(g, n[j][k], aw[j][k]);
                ab[j][k] += g;
                t[j][k] = g * wv[j][k];
                p += t[j][k];
                q = fmaf(t[j][k], n[j][k], q);
            }
            if (dres) cd[j] = rd[j];
        }
        if (row + step < M) fetch(row + step);
        row_sum2<TPR>(p, q, red[turn]);
        p /= (float)D;   // (not times 1 / D, whose rounding equal terms would keep, an ulp of theirs)
        q /= (float)D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPR + tid) * kNormVec;
            float o[kNormVec];
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                o[k] = (t[j][k] - fmaf(n[j][k], q, p)) * rc;
                if (dres) o[k] += cd[j].get(k);
            }
            if (c < D) {
                norm_vec<S, NT>::store(ds + row * D, c, D, o);
                if (dx) norm_vec<IO, NT>::store(dx + row * D, c, D, o);
            }
        }
    }
    if (!pw) return;
    if constexpr (SLOTS > 1) {   // the slots' sums, in order
        __shared__ float acc[2][NV * kNormVec][TPR];
        for (int k = SLOTS - 1; k >= 0; --k) {
            if (slot == k) {
#pragma unroll
                for (int j = 0; j < NV * kNormVec; ++j) {
                    if (k < SLOTS - 1) {
                        aw[j / kNormVec][j % kNormVec] += acc[0][j][tid];
                        ab[j / kNormVec][j % kNormVec] += acc[1][j][tid];
                    }
                    acc[0][j][tid] = aw[j / kNormVec][j % kNormVec];
                    acc[1][j][tid] = ab[j / kNormVec][j % kNormVec];
                }
            }
            __syncthreads();
        }
    }
    if (slot == 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPR + tid) * kNormVec;
#pragma unroll
            for (int k = 0; k < kNormVec; ++k)
                if (c + k < D) {
                    pw[(int64_t)blockIdx.x * D + c + k] = aw[j][k];
                    pb[(int64_t)blockIdx.x * D + c + k] = ab[j][k];
                }
        }
    }
}

// out[d] = sum of the n rows of each part, in an order of their own: kNormSumGroups groups of threads
// take every kNormSumGroups-th row of kNormSumCols columns, and their sums are added in order.  Bound:
// the latency of a few dependent loads (512 parts of 1536 columns: 3.9 us).
constexpr int kNormSumCols = 32, kNormSumGroups = 32;
static __global__ void __launch_bounds__(kNormSumCols * kNormSumGroups)
layernorm_wgrad_sum_kernel(const float *__restrict__ pw, const float *__restrict__ pb, float *__restrict__ dw,
                           float *__restrict__ db, int64_t n, int64_t D) {
    __shared__ float red[2][kNormSumGroups][kNormSumCols];
    const int col = threadIdx.x % kNormSumCols, g = threadIdx.x / kNormSumCols;
    const int64_t d = (int64_t)blockIdx.x * kNormSumCols + col;
    float a = 0.0f, b = 0.0f;
    if (d < D) {
#pragma unroll 8
        for (int64_t k = g; k < n; k += kNormSumGroups) {
            a += pw[k * D + d];
            b += pb[k * D + d];
        }
    }
    red[0][g][col] = a;
    red[1][g][col] = b;
    __syncthreads();
    if (g < 2 && d < D) {
        float t = red[g][0][col];
#pragma unroll
        for (int k = 1; k < kNormSumGroups; ++k) t += red[g][k][col];
        float *o = g == 0 ? dw : db;
        if (o) o[d] = t;
    }
}

// ---- rows wider than the registers hold: one workgroup per row, several passes over it ----------
// (2048x20000 bf16 with fp32 sums: 138 us for 492 MB; 4096x8200, the backward: 119 us for 537 MB and 46
// for the parameters' sums, which read dy and s once more.)

constexpr int kNormWideThreads = 1024;
constexpr int kNormWideStep = kNormWideThreads * kNormVec;

template <typename IO, typename S>
__global__ void __launch_bounds__(kNormWideThreads)
layernorm_fwd_wide_kernel(const IO *__restrict__ x, const S *res, const float *__restrict__ w,
                          const float *__restrict__ bias, float eps, IO *__restrict__ y, S *sum,
                          float *__restrict__ mean, float *__restrict__ rstd, int64_t M, int64_t D) {
    __shared__ float red[kNormWideThreads / 64], red2[kNormWideThreads / 64][2];
    const float inv_d = 1.0f / (float)D;
    const int64_t c0 = threadIdx.x * kNormVec;
    for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
        const int64_t o = row * D;
        auto values = [&](int64_t c, float (&v)[kNormVec]) {   // (0 past the row's end)
            norm_vec<IO, false> rx;
            norm_vec<S, false> rr;
            rx.load(x + o, c, D);
            if (res) rr.load(res + o, c, D);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                v[k] = rx.get(k);
                if (res) v[k] += rr.get(k);
                if constexpr (sizeof(S) == 2) v[k] = bf16_to_f32(f32_to_bf16(v[k]));
            }
        };
        float m = 0.0f, e = 0.0f, q = 0.0f, v[kNormVec];
        for (int64_t c = c0; c < D; c += kNormWideStep) {
            values(c, v);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) m += v[k];
        }
        m = row_sum<kNormWideThreads>(m, red) * inv_d;
        for (int64_t c = c0; c < D; c += kNormWideStep) {
            values(c, v);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                const float t = c + k < D ? v[k] - m : 0.0f;
                e += t;
                q = fmaf(t, t, q);
            }
        }
        row_sum2<kNormWideThreads>(e, q, red2);
        e *= inv_d;
        const float rs = rstd_of(q, inv_d, e, eps), shift = -e * rs;
        for (int64_t c = c0; c < D; c += kNormWideStep) {
            float wv[kNormVec], bv[kNormVec], n[kNormVec];
            values(c, v);
            load_params(w, c, D, wv);
            load_params(bias, c, D, bv);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) n[k] = fmaf(fmaf(v[k] - m, rs, shift), wv[k], bv[k]);
            if (sum) norm_vec<S, false>::store(sum + o, c, D, v);
            norm_vec<IO, false>::store(y + o, c, D, n);
        }
        if (threadIdx.x == 0) {
            if (mean) mean[row] = m + e;
            if (rstd) rstd[row] = rs;
        }
    }
}

template <typename IO, typename S>
__global__ void __launch_bounds__(kNormWideThreads)
layernorm_bwd_wide_kernel(const IO *__restrict__ dy, const S *__restrict__ s, const float *__restrict__ w,
                          const float *__restrict__ mean, const float *__restrict__ rstd, const S *dres, S *ds,
                          IO *__restrict__ dx, int64_t M, int64_t D) {
    __shared__ float red[2][kNormWideThreads / 64][2];
    const int64_t c0 = threadIdx.x * kNormVec;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < M; row += gridDim.x, turn ^= 1) {
        const int64_t o = row * D;
        const float m = mean[row], rs = rstd[row];
        auto values = [&](int64_t c, float (&t)[kNormVec], float (&n)[kNormVec]) {   // dy w and n
            norm_vec<IO, false> rg;
            norm_vec<S, false> rv;
            float wv[kNormVec];
            rg.load(dy + o, c, D);
            rv.load(s + o, c, D);
            load_params(w, c, D, wv);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                t[k] = rg.get(k) * wv[k];
                n[k] = c + k < D ? (rv.get(k) - m) * rs : 0.0f;
            }
        };
        float p = 0.0f, q = 0.0f, t[kNormVec], n[kNormVec];
        for (int64_t c = c0; c < D; c += kNormWideStep) {
            values(c, t, n);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                p += t[k];
                q = fmaf(t[k], n[k], q);
            }
        }
        row_sum2<kNormWideThreads>(p, q, red[turn]);
        p /= (float)D;   // (not times 1 / D, whose rounding equal terms would keep, an ulp of theirs)
        q /= (float)D;
        for (int64_t c = c0; c < D; c += kNormWideStep) {
            norm_vec<S, false> rd;
            values(c, t, n);
            if (dres) rd.load(dres + o, c, D);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                t[k] = (t[k] - fmaf(n[k], q, p)) * rs;
                if (dres) t[k] += rd.get(k);
            }
            norm_vec<S, false>::store(ds + o, c, D, t);
            if (dx) norm_vec<IO, false>::store(dx + o, c, D, t);
        }
    }
}

// The parameters' gradients over rows [blockIdx.y * rows_per, ...), kNormVec columns per thread.
template <typename IO, typename S>
__global__ void __launch_bounds__(256)
layernorm_wgrad_wide_kernel(const IO *__restrict__ dy, const S *__restrict__ s, const float *__restrict__ mean,
                            const float *__restrict__ rstd, float *__restrict__ pw, float *__restrict__ pb, int64_t M,
                            int64_t D, int64_t rows_per) {
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * kNormVec;
    if (c >= D) return;
    const int64_t r1 = min(M, (blockIdx.y + 1) * rows_per);
    float a[kNormVec] = {}, b[kNormVec] = {};
#pragma unroll 4
    for (int64_t i = blockIdx.y * rows_per; i < r1; ++i) {
        norm_vec<IO, false> rg;
        norm_vec<S, false> rv;
        rg.load(dy + i * D, c, D);
        rv.load(s + i * D, c, D);
#pragma unroll
        for (int k = 0; k < kNormVec; ++k) {
            a[k] = fmaf(rg.get(k), (rv.get(k) - mean[i]) * rstd[i], a[k]);
            b[k] += rg.get(k);
        }
    }
    norm_vec<float, false>::store(pw + blockIdx.y * D, c, D, a);
    norm_vec<float, false>::store(pb + blockIdx.y * D, c, D, b);
}

}  // namespace ssm
