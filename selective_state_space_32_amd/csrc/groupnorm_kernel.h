// Group norm over the channels of a row, channels last, with an activation, and its gradients.  A row of
// C values is G groups of D = C / G; per row and group
//
//   v = x silu(z) (gate first) or x;   mu = mean(v) (0 without centring),  rstd = 1 / sqrt(mean((v - mu)^2) + eps)
//   n = (v - mu) rstd,   o = n w + b,   y = o, or o silu(z) (gate after), or silu(o)
//   with do = dy d y / d o and dn = do w:   dv = rstd (dn - mean(dn) (with centring) - n mean(dn n))
//   dw = sum over rows of do n,   db = sum over rows of do
//
// Bound: HBM (x, z and dy are read once, y, dx and dz written once).  A group's values live in the registers
// of TPG threads, NV vectors of kNormVec each: 8 lanes for groups of 32, a wave for up to 1024, a workgroup
// beyond.  A thread keeps its columns over all the rows that its workgroup takes, so that the weights stay
// in registers, and so do the sums over rows behind dw and db.  Groups wider than the registers hold are
// passed over several times.  The activation is the kernel's, not the launch's: when it became so, 16384x5120 bf16 of 8
// groups, gate first, went from 128 to 120 us, its backward from 302 to 262.
// Measured: that case 102 us (503 MB, 4.9 TB/s), backward 191 + 5 us (839 MB, 4.3 TB/s); 4096x1536 fp32 of
// groups of 64, gate after, 14.4 and 23 + 4 us; 256x5120 bf16, one group, 6.0 us.
#pragma once

#include "layernorm_kernel.h"

namespace ssm {

constexpr int kGnPlain = 0, kGnGateFirst = 1, kGnGateAfter = 2, kGnSilu = 3;

// Where a launch's workgroups find their work: `spr` groups of a row side by side, `rpb` rows at a time,
// `gblocks` workgroups across a row.
struct gn_shape {
    int64_t M, C, D, zs;    // rows, channels, channels per group, elements between rows of z
    int G, spr, rpb, gblocks, act, centre;   // act: the kernels' ACT
};

// A product that is rounded before a mean is taken from it: fused into the difference it would not be the value whose
// mean was taken (a group of one channel has n = 0 and dx = 0).
__device__ __forceinline__ float product(float a, float b) {
#pragma clang fp contract(off)
    return a * b;
}

template <int TPG> __device__ __forceinline__ float group_sum(float p, float *red) {
    if constexpr (TPG > 64) return row_sum<TPG>(p, red);
    else return lanes_sum<TPG>(p);
}
template <int TPG> __device__ __forceinline__ void group_sum2(float &p, float &q, float (*red)[2]) {
    if constexpr (TPG > 64) {
        row_sum2<TPG>(p, q, red);
    } else {
        p = lanes_sum<TPG>(p);
        q = lanes_sum<TPG>(q);
    }
}

template <int TPG> constexpr int gn_threads() { return TPG > 256 ? TPG : 256; }

// The thread's group and rows: `g` and the first row, or no rows (its slot has no group).
template <int TPG> struct gn_place {
    int g, tid;
    int64_t row, step, part;
    bool has;
    __device__ __forceinline__ explicit gn_place(const gn_shape &s) {
        const int slot = TPG >= gn_threads<TPG>() ? 0 : threadIdx.x / TPG, sub = slot / s.spr;
        tid = threadIdx.x % TPG;
        g = blockIdx.x % s.gblocks * s.spr + slot - sub * s.spr;
        has = sub < s.rpb && g < s.G;
        part = (int64_t)(blockIdx.x / s.gblocks) * s.rpb + sub;
        step = (int64_t)(gridDim.x / s.gblocks) * s.rpb;
        row = has ? part : s.M;
        if (!has) g = 0;
    }
};

// (Lanes of a wave may run out of rows at different times: they exchange values within a group's lanes only.)
template <typename IO, int TPG, int NV, int ACT>
__global__ void __launch_bounds__(gn_threads<TPG>())
groupnorm_fwd_kernel(const IO *__restrict__ x, const IO *__restrict__ z, const float *__restrict__ w,
                     const float *__restrict__ bias, float eps, IO *__restrict__ y, float *__restrict__ mean,
                     float *__restrict__ rstd, gn_shape s) {
    using vec_t = norm_vec<IO, false>;
    constexpr bool kGated = ACT == kGnGateFirst || ACT == kGnGateAfter;
    __shared__ float red[TPG > 64 ? TPG / 64 : 1], red2[2][TPG > 64 ? TPG / 64 : 1][2];
    const gn_place<TPG> at(s);
    const int64_t c0 = (int64_t)at.g * s.D;
    const float inv_d = 1.0f / (float)s.D;
    float wv[NV][kNormVec], bv[NV][kNormVec];
    vec_t rx[NV], rz[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)(j * TPG + at.tid) * kNormVec;
        load_params(w + c0, c, s.D, wv[j]);
        load_params(bias ? bias + c0 : nullptr, c, s.D, bv[j]);
    }
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPG + at.tid) * kNormVec;
            rx[j].load(x + row * s.C + c0, c, s.D);
            if (kGated) rz[j].load(z + row * s.zs + c0, c, s.D);
        }
    };
    if (at.row < s.M) fetch(at.row);
    int turn = 0;   // (without centring this sum alone separates the rows: two sets of slots)
    for (int64_t row = at.row; row < s.M; row += at.step, turn ^= 1) {
        float v[NV][kNormVec], gate[NV][kNormVec];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                v[j][k] = rx[j].get(k);
                gate[j][k] = kGated ? silu_f32(rz[j].get(k)) : 1.0f;
                if (ACT == kGnGateFirst) v[j][k] = product(v[j][k], gate[j][k]);
            }
        if (row + at.step < s.M) fetch(row + at.step);
        float m = 0.0f, e = 0.0f, q = 0.0f;
        if (s.centre) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int k = 0; k < kNormVec; ++k) m += v[j][k];
            m = group_sum<TPG>(m, red) * inv_d;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPG + at.tid) * kNormVec;
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                v[j][k] = c + k < s.D ? v[j][k] - m : 0.0f;
                e += v[j][k];
                q = fmaf(v[j][k], v[j][k], q);
            }
        }
        group_sum2<TPG>(e, q, red2[turn]);
        e = s.centre ? e * inv_d : 0.0f;   // what the mean lacks (the sum's roundings)
        const float rs = rstd_of(q, inv_d, e, eps), shift = -e * rs;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPG + at.tid) * kNormVec;
            float o[kNormVec];
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                o[k] = fmaf(fmaf(v[j][k], rs, shift), wv[j][k], bv[j][k]);
                if (ACT == kGnGateAfter) o[k] *= gate[j][k];
                if (ACT == kGnSilu) o[k] = silu_f32(o[k]);
            }
            if (c < s.D) vec_t::store(y + row * s.C + c0, c, s.D, o);
        }
        if (at.tid == 0) {
            if (mean) mean[row * s.G + at.g] = m + e;
            if (rstd) rstd[row * s.G + at.g] = rs;
        }
    }
}

// The parts of a gradient that go by element: from x, z, dy and the statistics, do, n and (gate after) dz.
struct gn_elem {
    float dov, n, gate, dgate;   // d L / d o, the normalised value, silu(z) and its derivative
    float dz_after;              // gate after: dy o silu'(z)
};
__device__ __forceinline__ gn_elem gn_element(float x, float z, float dy, float w, float b, float m, float rs, int act) {
    gn_elem r;
    r.gate = 1.0f;
    r.dgate = r.dz_after = 0.0f;
    if (act == kGnGateFirst || act == kGnGateAfter) {
        const float sg = sigmoid_f32(z);
        r.gate = z * sg;
        r.dgate = sg * fmaf(z, 1.0f - sg, 1.0f);
    }
    const float v = act == kGnGateFirst ? product(x, r.gate) : x;
    r.n = (v - m) * rs;
    r.dov = dy;
    if (act == kGnGateAfter) {
        r.dz_after = dy * fmaf(r.n, w, b) * r.dgate;
        r.dov = dy * r.gate;
    } else if (act == kGnSilu) {
        const float o = fmaf(r.n, w, b), sg = sigmoid_f32(o);
        r.dov = dy * sg * fmaf(o, 1.0f - sg, 1.0f);
    }
    return r;
}

// pw, pb: [parts][C] sums over the rows of a part, or null.
template <typename IO, int TPG, int NV, int ACT>
__global__ void __launch_bounds__(gn_threads<TPG>()) __attribute__((amdgpu_waves_per_eu(NV <= 3 ? 4 : 2)))
groupnorm_bwd_kernel(const IO *__restrict__ dy, const IO *__restrict__ x, const IO *__restrict__ z,
                     const float *__restrict__ w, const float *__restrict__ bias, const float *__restrict__ mean,
                     const float *__restrict__ rstd, IO *__restrict__ dx, IO *__restrict__ dz, float *__restrict__ pw,
                     float *__restrict__ pb, gn_shape s) {
    using vec_t = norm_vec<IO, false>;
    constexpr bool kGated = ACT == kGnGateFirst || ACT == kGnGateAfter;
    __shared__ float red[2][TPG > 64 ? TPG / 64 : 1][2];
    const gn_place<TPG> at(s);
    const int64_t c0 = (int64_t)at.g * s.D;
    float wv[NV][kNormVec], bv[NV][kNormVec], aw[NV][kNormVec] = {}, ab[NV][kNormVec] = {};
    vec_t rx[NV], rz[NV], rg[NV];
    float m = 0.0f, rs = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)(j * TPG + at.tid) * kNormVec;
        load_params(w + c0, c, s.D, wv[j]);
        load_params(bias ? bias + c0 : nullptr, c, s.D, bv[j]);
    }
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPG + at.tid) * kNormVec;
            rx[j].load(x + row * s.C + c0, c, s.D);
            rg[j].load(dy + row * s.C + c0, c, s.D);
            if (kGated) rz[j].load(z + row * s.zs + c0, c, s.D);
        }
        m = s.centre ? mean[row * s.G + at.g] : 0.0f;
        rs = rstd[row * s.G + at.g];
    };
    if (at.row < s.M) fetch(at.row);
    int turn = 0;
    for (int64_t row = at.row; row < s.M; row += at.step, turn ^= 1) {
        // The row is held as it was read and its elements are formed twice, before and after the sums.  (That the compiler
        // may hold the first ones instead, as far as the waves that are asked for leave registers, costs nothing: with an
        // empty asm against it 16384x5120 bf16 of 8 groups takes 195 us gate first, 194 without, 197 and 181 gate after.)
        vec_t nx[NV], nz[NV], ng[NV];
        const float m_now = m, rs_now = rs;
        float p = 0.0f, q = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPG + at.tid) * kNormVec;
            nx[j] = rx[j];
            ng[j] = rg[j];
            if (kGated) nz[j] = rz[j];
            float za[kNormVec];
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                const bool in = c + k < s.D;
                const gn_elem el = gn_element(rx[j].get(k), kGated ? rz[j].get(k) : 0.0f, rg[j].get(k), wv[j][k], bv[j][k], m, rs, ACT);
                const float dn = product(el.dov, wv[j][k]);
                za[k] = el.dz_after;
                if (in) {
                    aw[j][k] = fmaf(el.dov, el.n, aw[j][k]);
                    ab[j][k] += el.dov;
                    p += dn;
                    q = fmaf(dn, el.n, q);
                }
            }
            if (ACT == kGnGateAfter && c < s.D) vec_t::store(dz + row * s.C + c0, c, s.D, za);
        }
        if (row + at.step < s.M) fetch(row + at.step);
        group_sum2<TPG>(p, q, red[turn]);
        p = s.centre ? p / (float)s.D : 0.0f;
        q /= (float)s.D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPG + at.tid) * kNormVec;
            float o[kNormVec], oz[kNormVec];
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                const gn_elem el = gn_element(nx[j].get(k), kGated ? nz[j].get(k) : 0.0f, ng[j].get(k), wv[j][k], bv[j][k], m_now, rs_now, ACT);
                const float dv = (product(el.dov, wv[j][k]) - fmaf(el.n, q, p)) * rs_now;
                o[k] = ACT == kGnGateFirst ? dv * el.gate : dv;
                oz[k] = dv * nx[j].get(k) * el.dgate;
            }
            if (c < s.D) {
                vec_t::store(dx + row * s.C + c0, c, s.D, o);
                if (ACT == kGnGateFirst) vec_t::store(dz + row * s.C + c0, c, s.D, oz);
            }
        }
    }
    if (pw && at.has) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)(j * TPG + at.tid) * kNormVec;
            if (c < s.D) {
                norm_vec<float, false>::store(pw + at.part * s.C + c0, c, s.D, aw[j]);
                norm_vec<float, false>::store(pb + at.part * s.C + c0, c, s.D, ab[j]);
            }
        }
    }
}

// ---- groups wider than the registers hold: a workgroup per row and group, several passes over it --------

template <typename IO>
__global__ void __launch_bounds__(kNormWideThreads)
groupnorm_fwd_wide_kernel(const IO *__restrict__ x, const IO *__restrict__ z, const float *__restrict__ w,
                          const float *__restrict__ bias, float eps, IO *__restrict__ y, float *__restrict__ mean,
                          float *__restrict__ rstd, gn_shape s) {
    __shared__ float red[kNormWideThreads / 64], red2[kNormWideThreads / 64][2];
    const float inv_d = 1.0f / (float)s.D;
    const int64_t first = threadIdx.x * kNormVec;
    for (int64_t unit = blockIdx.x; unit < s.M * s.G; unit += gridDim.x) {
        const int64_t row = unit / s.G, c0 = (unit - row * s.G) * s.D;
        auto values = [&](int64_t c, float (&v)[kNormVec], float (&gate)[kNormVec]) {   // (0 past the group's end)
            norm_vec<IO, false> rx, rz;
            rx.load(x + row * s.C + c0, c, s.D);
            if (z) rz.load(z + row * s.zs + c0, c, s.D);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                gate[k] = z ? silu_f32(rz.get(k)) : 1.0f;
                v[k] = rx.get(k);
                if (s.act == kGnGateFirst) v[k] = product(v[k], gate[k]);
            }
        };
        float m = 0.0f, e = 0.0f, q = 0.0f, v[kNormVec], gate[kNormVec];
        if (s.centre) {
            for (int64_t c = first; c < s.D; c += kNormWideStep) {
                values(c, v, gate);
#pragma unroll
                for (int k = 0; k < kNormVec; ++k) m += v[k];
            }
            m = row_sum<kNormWideThreads>(m, red) * inv_d;
        }
        for (int64_t c = first; c < s.D; c += kNormWideStep) {
            values(c, v, gate);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                const float t = c + k < s.D ? v[k] - m : 0.0f;
                e += t;
                q = fmaf(t, t, q);
            }
        }
        row_sum2<kNormWideThreads>(e, q, red2);
        __syncthreads();   // (without centring nothing else separates this sum from the next unit's)
        e = s.centre ? e * inv_d : 0.0f;
        const float rs = rstd_of(q, inv_d, e, eps), shift = -e * rs;
        for (int64_t c = first; c < s.D; c += kNormWideStep) {
            float wv[kNormVec], bv[kNormVec], o[kNormVec];
            values(c, v, gate);
            load_params(w + c0, c, s.D, wv);
            load_params(bias ? bias + c0 : nullptr, c, s.D, bv);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                o[k] = fmaf(fmaf(v[k] - m, rs, shift), wv[k], bv[k]);
                if (s.act == kGnGateAfter) o[k] *= gate[k];
                if (s.act == kGnSilu) o[k] = silu_f32(o[k]);
            }
            norm_vec<IO, false>::store(y + row * s.C + c0, c, s.D, o);
        }
        if (threadIdx.x == 0) {
            if (mean) mean[unit] = m + e;
            if (rstd) rstd[unit] = rs;
        }
    }
}

template <typename IO>
__global__ void __launch_bounds__(kNormWideThreads)
groupnorm_bwd_wide_kernel(const IO *__restrict__ dy, const IO *__restrict__ x, const IO *__restrict__ z,
                          const float *__restrict__ w, const float *__restrict__ bias, const float *__restrict__ mean,
                          const float *__restrict__ rstd, IO *__restrict__ dx, IO *__restrict__ dz, gn_shape s) {
    __shared__ float red[2][kNormWideThreads / 64][2];
    const int64_t first = threadIdx.x * kNormVec;
    int turn = 0;
    for (int64_t unit = blockIdx.x; unit < s.M * s.G; unit += gridDim.x, turn ^= 1) {
        const int64_t row = unit / s.G, c0 = (unit - row * s.G) * s.D, o = row * s.C + c0;
        const float m = s.centre ? mean[unit] : 0.0f, rs = rstd[unit];
        float p = 0.0f, q = 0.0f;
        auto elements = [&](int64_t c, float (&wv)[kNormVec], float (&xv)[kNormVec], gn_elem (&el)[kNormVec]) {
            norm_vec<IO, false> rx, rz, rg;
            float bv[kNormVec];
            rx.load(x + o, c, s.D);
            rg.load(dy + o, c, s.D);
            if (z) rz.load(z + row * s.zs + c0, c, s.D);
            load_params(w + c0, c, s.D, wv);
            load_params(bias ? bias + c0 : nullptr, c, s.D, bv);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                xv[k] = rx.get(k);
                el[k] = gn_element(xv[k], z ? rz.get(k) : 0.0f, rg.get(k), wv[k], bv[k], m, rs, s.act);
            }
        };
        for (int64_t c = first; c < s.D; c += kNormWideStep) {
            float wv[kNormVec], xv[kNormVec];
            gn_elem el[kNormVec];
            elements(c, wv, xv, el);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                const float t = c + k < s.D ? product(el[k].dov, wv[k]) : 0.0f;
                p += t;
                if (c + k < s.D) q = fmaf(t, el[k].n, q);
            }
        }
        row_sum2<kNormWideThreads>(p, q, red[turn]);
        p = s.centre ? p / (float)s.D : 0.0f;
        q /= (float)s.D;
        for (int64_t c = first; c < s.D; c += kNormWideStep) {
            float wv[kNormVec], xv[kNormVec], ox[kNormVec], oz[kNormVec];
            gn_elem el[kNormVec];
            elements(c, wv, xv, el);
#pragma unroll
            for (int k = 0; k < kNormVec; ++k) {
                const float dv = (product(el[k].dov, wv[k]) - fmaf(el[k].n, q, p)) * rs;
                ox[k] = s.act == kGnGateFirst ? dv * el[k].gate : dv;
                oz[k] = s.act == kGnGateFirst ? dv * xv[k] * el[k].dgate : el[k].dz_after;
            }
            norm_vec<IO, false>::store(dx + o, c, s.D, ox);
            if (z) norm_vec<IO, false>::store(dz + o, c, s.D, oz);
        }
    }
}

// The parameters' gradients over rows [blockIdx.y * rows_per, ...), kNormVec columns of one group per thread.
template <typename IO>
__global__ void __launch_bounds__(256)
groupnorm_wgrad_wide_kernel(const IO *__restrict__ dy, const IO *__restrict__ x, const IO *__restrict__ z,
                            const float *__restrict__ w, const float *__restrict__ bias, const float *__restrict__ mean,
                            const float *__restrict__ rstd, float *__restrict__ pw, float *__restrict__ pb, gn_shape s,
                            int64_t rows_per) {
    const int64_t vecs = (s.D + kNormVec - 1) / kNormVec, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t g = id / vecs, c = (id - g * vecs) * kNormVec, c0 = g * s.D;
    if (g >= s.G) return;
    const int64_t r1 = min(s.M, (blockIdx.y + 1) * rows_per);
    float a[kNormVec] = {}, b[kNormVec] = {}, wv[kNormVec], bv[kNormVec];
    load_params(w + c0, c, s.D, wv);
    load_params(bias ? bias + c0 : nullptr, c, s.D, bv);
    for (int64_t i = blockIdx.y * rows_per; i < r1; ++i) {
        norm_vec<IO, false> rx, rz, rg;
        rx.load(x + i * s.C + c0, c, s.D);
        rg.load(dy + i * s.C + c0, c, s.D);
        if (z) rz.load(z + i * s.zs + c0, c, s.D);
        const float m = s.centre ? mean[i * s.G + g] : 0.0f, rs = rstd[i * s.G + g];
#pragma unroll
        for (int k = 0; k < kNormVec; ++k) {
            const gn_elem el = gn_element(rx.get(k), z ? rz.get(k) : 0.0f, rg.get(k), wv[k], bv[k], m, rs, s.act);
            a[k] = fmaf(el.dov, el.n, a[k]);
            b[k] += el.dov;
        }
    }
    norm_vec<float, false>::store(pw + blockIdx.y * s.C + c0, c, s.D, a);
    norm_vec<float, false>::store(pb + blockIdx.y * s.C + c0, c, s.D, b);
}

}  // namespace ssm
