// Gradients of the state space dual layer with its convolution (ssd_conv_kernel.h has its operands and
// tiles).  With ds_c the adjoint of the state leaving a chunk and S the state entering it, T = dy x^T:
//   v_s   = sum_{t >= s} G[t,s] K[t,s] dy_t + e^{c_last - c_s} dS B_s
//   dx_s  = dt_s v_s + D dy_s
//   Z     = T K dt (summed over a group's heads),   dB = Z^T C + sum_h e^{c_last - c_s} dt_s dS^T x_s
//                                                   dC = Z B   + sum_h e^{c_t} S^T dy_t
//   dS entering = e^{c_last} dS + sum_t e^{c_t} dy_t C_t^T
// and for the step sizes, with W = G T K dt below the diagonal (t > s),
//   q_s  = v_s . x_s
//   dg_s = sum_{t >= s > r} W[t,r] + sum_{t >= s} e^{c_t} dy_t . S C_t + sum_{r < s} e^{c_last - c_r} dt_r x_r . dS B_r
//          + e^{c_last} <dS, S>
//   ddt_s = q_s + A dg_s,   dA = sum dt_s dg_s,   dD = sum dy . x
// (dg_s is the gradient of the logarithm of token s's decay: the paths from before s to s or later.  The first sum
// is suffix sums of W's rows less those of its columns, in 64 bits.)
#pragma once

#include "ssd_conv_kernel.h"
#include "wave_sum.h"

namespace ssm {

// The states entering the chunks (ADJ = false: rows x, weights e^{c_last - c} dt, with B) or the adjoints of the
// states leaving them (ADJ: rows dy, weights e^c, with C, chunks from the last), one workgroup per (sequence, head,
// 64-channel tile, segment).  each: [b][h][chunk][P][N], or null.  from: [b][h][segment][P][N], or null (zero).  to: with
// `ends` [b][h][segment][P][N], what every segment leaves, else [b][h][P][N], what the last (ADJ: first) one leaves, or null.
template <typename E, int NT, bool ADJ>
__global__ void __launch_bounds__(kSdThreads)
sd_walk_kernel(const typename sd<E>::io *__restrict__ u_, const typename sd<E>::io *__restrict__ dy_,
               const float *__restrict__ tok, const int32_t *__restrict__ lens, const float *__restrict__ from, float *__restrict__ each,
               float *__restrict__ to, int ends, sd_shape s) {
    using IO = typename sd<E>::io;
    using F = typename sd<E>::frag;
    constexpr int NB = NT / 16;
    __shared__ __attribute__((aligned(16))) E tB[64 * sd_ld<E>(NT)], tX[64 * sd_ld<E>(64)];
    __shared__ sd_tokens tk;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q4 = 4 * (lane >> 4);
    const sd_segment at(s, lens);
    const int64_t b = at.b, len = at.len;
    const int h = at.h, pt = at.pt;
    const sd_view<IO> v(u_, s, b, h, pt);
    const int xrow = ADJ ? s.H * s.P : s.dc;
    const E *xs = reinterpret_cast<const E *>(ADJ ? dy_ + (b * s.L * s.H + h) * s.P + pt * 64 : v.x);
    const E *Bs = reinterpret_cast<const E *>(ADJ ? v.C : v.B);
    tok += (b * s.H + h) * s.nchunk * kSdTok;
    f32x4_t S[NB];
    if (from) {
        sd_load_state(S, from + at.state_at(s, s.nseg, at.seg), s.N, v.pw, w, lane);
    } else {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    auto keep = [&](int64_t c) {
        if (each) sd_store_state(S, each + at.state_at(s, s.nchunk, c), s.N, v.pw, w, lane);
    };
    if (ADJ)   // chunks past the sequence's end leave the adjoint as it is
        for (int64_t c = at.live; c < at.c1; ++c) keep(c);
    tile64<E, NT> rB;
    tile64<E, 64> rX;
    sd_tok rt = {};
    auto fetch = [&](int64_t c) {
        const int64_t t0 = c * kSdQ;
        const int rows = (int)min((int64_t)64, len - t0);
        rB.load(Bs + t0 * s.dc, s.dc, rows, s.N);
        rX.load(xs + t0 * xrow, (uint32_t)xrow, rows, v.pw);
        if (w == 0) rt = sd_load_tokens(tok + c * kSdTok, lane);
    };
    const int64_t n = at.live - at.c0;
    if (n > 0) fetch(ADJ ? at.live - 1 : at.c0);
    for (int64_t i = 0; i < n; ++i) {
        const int64_t c = ADJ ? at.live - 1 - i : at.c0 + i;
        rB.stage(tB);
        rX.stage(tX);
        if (w == 0) sd_stage_tokens(tk, rt, lane);
        if (i + 1 < n) fetch(ADJ ? c - 1 : c + 1);
        keep(c);
        __syncthreads();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb] *= tk.dec;
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
            const float *wt = (ADJ ? tk.e : tk.w) + 16 * k + q4;
            const F x0 = ld_col<E, 64>(tX, 16 * k, 16 * w, lane), x1 = ld_col<E, 64>(tX, 16 * k + 16, 16 * w, lane);
            const formed<E, 3> f0(widen(x0) * ld4(wt)), f1(widen(x1) * ld4(wt + 16));
#pragma unroll
            for (int n0 = 0; n0 < NB; n0 += 4) {
                F b0[4], b1[4];
#pragma unroll
                for (int nb = 0; nb < 4; ++nb) {
                    b0[nb] = ld_col<E, NT>(tB, 16 * k, 16 * (n0 + nb), lane);
                    b1[nb] = ld_col<E, NT>(tB, 16 * k + 16, 16 * (n0 + nb), lane);
                }
#pragma unroll
                for (int m = 0; m < formed<E, 3>::N; ++m)
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb) S[n0 + nb] = mma(b0[nb], b1[nb], f0.p[m], f1.p[m], S[n0 + nb]);
            }
        }
        __syncthreads();
    }
    if (!ADJ)
        for (int64_t c = at.live; c < at.c1; ++c) keep(c);
    if (ends) sd_store_state(S, to + at.state_at(s, s.nseg, at.seg), s.N, v.pw, w, lane);
    else if (to && at.seg == (ADJ ? 0 : s.nseg - 1)) sd_store_state(S, to + at.state_at(s, 1, 0), s.N, v.pw, w, lane);
}

// 64 x 64 of a state [p][n] in fp32 from memory to LDS, as NS operand parts.
template <typename E, int NS> struct state64 {
    static constexpr int NP = formed<E, NS>::N;
    f32x4_t r[4];
    __device__ __forceinline__ void load(const float *m, int N, int pw, int nw) {   // N: row stride; pw x nw exist
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int id = threadIdx.x + kSdThreads * i, p = id / 16, n = id % 16 * 4;
            r[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            if (p < pw && n < nw) r[i] = ld4(m + (int64_t)p * N + n);
        }
    }
    __device__ __forceinline__ void stage(E (&t)[NP][64 * sd_ld<E>(64)]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int id = threadIdx.x + kSdThreads * i, p = id / 16, n = id % 16 * 4;
            const formed<E, NS> f(r[i]);
#pragma unroll
            for (int k = 0; k < NP; ++k) *reinterpret_cast<typename sd<E>::frag *>(&t[k][p * sd_ld<E>(64) + n]) = f.p[k];
        }
    }
    __device__ __forceinline__ float dot(const state64 &o) const {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) a = fmaf(r[i][e], o.r[i][e], a);
        return a;
    }
};
__device__ __forceinline__ double wave_last(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, 63), hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// sum over the four 16-lane rows of a wave, in every lane
__device__ __forceinline__ float quads_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

struct sd_grad {
    float *du;      // [b][t][H P], the x part of u's gradient
    float *dbc;     // [HS][b][t][2 G N], parts of B's and C's
    float *part;    // [b * chunk][3][H]: parts of dA, ddt_bias, dD
    int HS, hpw;    // parts of a group's heads; heads per part
};

// One workgroup per (chunk, sequence, group, part of its heads), the heads in turn.  Wave w owns the 16 tokens
// 16 w .. of the chunk (as s of T, G, v, dB and as t of dC).
template <typename E, int NT>
__global__ void __launch_bounds__(kSdThreads)
sd_bwd_kernel(const typename sd<E>::io *__restrict__ u_, const typename sd<E>::io *__restrict__ dy_,
              const float *__restrict__ tok, const typename sd<E>::io *__restrict__ dt, const float *__restrict__ A,
              const float *__restrict__ Dv, const float *__restrict__ dt_bias, const int32_t *__restrict__ lens,
              const float *__restrict__ st_in,
              const float *__restrict__ ds_out, typename sd<E>::io *__restrict__ ddt, sd_grad gr, sd_shape s) {
    using IO = typename sd<E>::io;
    using F = typename sd<E>::frag;
    constexpr int NB = NT / 16, NP = formed<E, 2>::N, LD = sd_ld<E>(64);
    __shared__ __attribute__((aligned(16))) E tB[64 * sd_ld<E>(NT)], tC[64 * sd_ld<E>(NT)], tX[64 * LD], tY[64 * LD];
    __shared__ __attribute__((aligned(16))) E tS[NP][64 * LD], tD[NP][64 * LD];
    __shared__ sd_tokens tk;
    __shared__ float to_end[64];                        // e^{c_last - c_t}
    __shared__ float sR[4][64], sCol[64], sYS[64], sXS[64], sQ[64], sXY[64], sDot[4];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, q4 = 4 * (lane >> 4), mine = 16 * w + c16;   // the lane's token of the wave's 16
    const int64_t chunk = blockIdx.x % s.nchunk, rest = blockIdx.x / s.nchunk;
    const int hs = rest % gr.HS, g = rest / gr.HS % s.G;
    const int64_t b = rest / gr.HS / s.G, t0 = chunk * kSdQ;
    const int per = s.H / s.G, h0 = g * per + hs * gr.hpw, h1 = min(h0 + gr.hpw, (g + 1) * per);
    const int64_t len = lens ? min(max((int64_t)lens[b], (int64_t)0), s.L) : s.L;
    const int rows = (int)min((int64_t)64, max(len - t0, (int64_t)0)), tokens = (int)min((int64_t)64, s.L - t0);
    const bool have = t0 + mine < s.L;
    const IO *ub = u_ + (b * s.L + t0) * s.dc, *dyb = dy_ + (b * s.L + t0) * s.H * s.P;
    {
        tile64<E, NT> rB, rC;
        const E *B = reinterpret_cast<const E *>(ub + s.H * s.P + g * s.N);
        rB.load(B, s.dc, rows, s.N);
        rC.load(B + s.G * s.N, s.dc, rows, s.N);
        rB.stage(tB);
        rC.stage(tC);
    }
    __syncthreads();
    f32x4_t G[4] = {}, Z[4] = {}, dB[NB] = {}, dC[NB] = {};
#pragma unroll
    for (int k = 0; k < NB; k += 2) {
        const F b0 = ld_row<E, NT>(tB, 16 * w, 16 * k, lane), b1 = ld_row<E, NT>(tB, 16 * w, 16 * k + 16, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i >= w) G[i] = mma(ld_row<E, NT>(tC, 16 * i, 16 * k, lane), ld_row<E, NT>(tC, 16 * i, 16 * k + 16, lane), b0, b1, G[i]);
    }
    for (int h = h0; h < h1; ++h) {
        const float a = A[h], skip = Dv ? Dv[h] : 0.0f;
        float rdt = 0.0f, sig = 0.0f;
        f32x4_t T[4] = {};
        float xs = 0.0f, ys = 0.0f, q = 0.0f, dot = 0.0f, xy = 0.0f;
        f32x4_t kk[4];
        for (int pt = 0; pt < s.PT; ++pt) {
            const int pw = min(64, s.P - pt * 64);
            const int64_t st_at = (((b * s.H + h) * s.nchunk + chunk) * s.P + (int64_t)pt * 64) * s.N;
            f32x4_t V[4] = {};
            F xf[4], yf[4];
            for (int nh = 0; nh < s.N; nh += 64) {   // 64 states at a time
                __syncthreads();
                if (nh == 0) {
                    tile64<E, 64> rX, rY;
                    rX.load(reinterpret_cast<const E *>(ub + h * s.P + pt * 64), s.dc, rows, pw);
                    rY.load(reinterpret_cast<const E *>(dyb + h * s.P + pt * 64), (uint32_t)(s.H * s.P), rows, pw);
                    rX.stage(tX);
                    rY.stage(tY);
                    if (pt == 0 && w == 0) {
                        const sd_tok rt = sd_load_tokens(tok + ((b * s.H + h) * s.nchunk + chunk) * kSdTok, lane);
                        to_end[lane] = sd_stage_tokens(tk, rt, lane);
                        rdt = rt.d;
                        sig = 0.0f;
                        if (lane < rows) {
                            sig = 1.0f;
                            if (s.softplus) softplus_f32(io<IO>::ld(dt, (b * s.L + t0 + lane) * s.dt_stride + h) + (dt_bias ? dt_bias[h] : 0.0f), sig);
                        }
                    }
                }
                state64<E, 2> rS, rD;
                rS.load(st_in + st_at + nh, s.N, pw, s.N - nh);
                rD.load(ds_out + st_at + nh, s.N, pw, s.N - nh);
                rS.stage(tS);
                rD.stage(tD);
                dot += rS.dot(rD);
                __syncthreads();
                const float et = tk.e[mine], ws = tk.w[mine];
                if (nh == 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        xf[i] = ld_row<E, 64>(tX, 16 * w, 16 * i, lane);
                        yf[i] = ld_row<E, 64>(tY, 16 * w, 16 * i, lane);
                    }
                    // T[t][s], rows t >= s only
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i >= w) {
#pragma unroll
                            for (int k = 0; k < 4; k += 2)
                                T[i] = mma(ld_row<E, 64>(tY, 16 * i, 16 * k, lane), ld_row<E, 64>(tY, 16 * i, 16 * k + 16, lane), xf[k], xf[k + 1], T[i]);
                        }
                    if (pt == 0) {
                        const float sh = tk.ch[mine], sl = tk.cl[mine];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            kk[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
                            if (i < w) continue;
                            const f32x4_t th = ld4(tk.ch + 16 * i + q4), tl = ld4(tk.cl + 16 * i + q4);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (16 * i + q4 + e >= mine) kk[i][e] = hw_exp2((th[e] - sh) + (tl[e] - sl));
                        }
                    }
                }
                // through the state leaving the chunk: V^T[p][s] and dB^T[n][s]; through the state entering: dC^T[n][t]
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    if (nh + 16 * k >= NT) continue;
                    const F b0 = ld_row<E, NT>(tB, 16 * w, nh + 16 * k, lane), b1 = ld_row<E, NT>(tB, 16 * w, nh + 16 * k + 16, lane);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int m = 0; m < NP; ++m)
                            V[j] = mma(ld_row<E, 64>(tD[m], 16 * j, 16 * k, lane), ld_row<E, 64>(tD[m], 16 * j, 16 * k + 16, lane), b0, b1, V[j]);
                }
#pragma unroll
                for (int half = 0; half < NT / 64; ++half) {
                    if (nh != 64 * half) continue;
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb) {
                        f32x4_t db = {}, dc = {};
#pragma unroll
                        for (int k = 0; k < 4; k += 2)
#pragma unroll
                            for (int m = 0; m < NP; ++m) {
                                db = mma(ld_col<E, 64>(tD[m], 16 * k, 16 * nb, lane), ld_col<E, 64>(tD[m], 16 * k + 16, 16 * nb, lane), xf[k], xf[k + 1], db);
                                dc = mma(ld_col<E, 64>(tS[m], 16 * k, 16 * nb, lane), ld_col<E, 64>(tS[m], 16 * k + 16, 16 * nb, lane), yf[k], yf[k + 1], dc);
                            }
                        const f32x4_t cf = widen(ld_row<E, NT>(tC, 16 * w, nh + 16 * nb, lane));
                        dc *= et;
                        dB[4 * half + nb] += db * ws;
                        dC[4 * half + nb] += dc;
                        ys += dc[0] * cf[0] + dc[1] * cf[1] + dc[2] * cf[2] + dc[3] * cf[3];
                    }
                }
            }
            {
                const float te = to_end[mine], d = tk.dt[mine];
                float x0 = 0.0f, q0 = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    V[j] *= te;
                    const f32x4_t x = widen(xf[j]), y = widen(yf[j]);
                    x0 += V[j][0] * x[0] + V[j][1] * x[1] + V[j][2] * x[2] + V[j][3] * x[3];
                    xy += x[0] * y[0] + x[1] * y[1] + x[2] * y[2] + x[3] * y[3];
                }
                xs += x0 * d;
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    if (i + 1 < w) continue;
                    const formed<E, 2> g0(G[i] * kk[i]), g1(G[i + 1] * kk[i + 1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        V[j] = mma_fb<E, 2>(ld_col<E, 64>(tY, 16 * i, 16 * j, lane), ld_col<E, 64>(tY, 16 * i + 16, 16 * j, lane), g0, g1, V[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4_t x = widen(xf[j]), y = widen(yf[j]);
                    q0 += V[j][0] * x[0] + V[j][1] * x[1] + V[j][2] * x[2] + V[j][3] * x[3];
                    if (have && 16 * j + q4 < pw)
                        *reinterpret_cast<f32x4_t *>(gr.du + ((b * s.L + t0 + mine) * s.H + h) * s.P + pt * 64 + 16 * j + q4) = V[j] * d + y * skip;
                }
                q += q0;
            }
        }
        // the head's sums over pairs of tokens
        const float d = tk.dt[mine];
        float col = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4_t z = T[i] * kk[i] * d;
            Z[i] += z;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 16 * i + q4 + e;
                const float wv = t > mine ? z[e] * G[i][e] : 0.0f;
                col += wv;
                const float r = lanes_sum<16>(wv);
                if (c16 == 0) sR[w][t] = r;
            }
        }
        col = quads_sum(col);
        xs = quads_sum(xs);
        ys = quads_sum(ys);
        q = quads_sum(q);
        xy = quads_sum(xy);
        dot = wave_sum(dot);
        if (lane < 16) {
            sCol[mine] = col;
            sXS[mine] = xs;
            sYS[mine] = ys;
            sQ[mine] = q;
            sXY[mine] = xy;
        }
        if (lane == 0) sDot[w] = dot;
        __syncthreads();
        if (w == 0) {   // token = lane
            const double v = (double)(sR[0][lane] + sR[1][lane] + sR[2][lane] + sR[3][lane]) - sCol[lane] + sYS[lane];
            const double p = wave_incl_sum64(v), x = sXS[lane], px = wave_incl_sum64(x);
            const double ends = (double)tk.dec * ((sDot[0] + sDot[1]) + (sDot[2] + sDot[3]));
            const float dg = (float)((wave_last(p) - p + v) + (px - x) + ends);
            const float dr = (sQ[lane] + a * dg) * sig;
            if (lane < tokens) io<IO>::st(ddt, (b * s.L + t0 + lane) * s.H + h, dr);
            const float pa = wave_sum(rdt * dg), pb = wave_sum(dr), pd = wave_sum(sXY[lane]);
            if (lane == 0) {
                float *o = gr.part + (b * s.nchunk + chunk) * 3 * s.H + h;
                o[0] = pa;
                o[s.H] = pb;
                o[2 * s.H] = pd;
            }
        }
    }
    // the products that the group's heads share: Z to LDS as [t][s] for dC, from registers for dB
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const formed<E, 2> f(Z[i]);
#pragma unroll
        for (int m = 0; m < NP; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) tS[m][(16 * i + q4 + e) * LD + mine] = f.p[m][e];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const formed<E, 2> z0(Z[i]), z1(Z[i + 1]);
        F r0[NP], r1[NP];
#pragma unroll
        for (int m = 0; m < NP; ++m) {
            r0[m] = ld_row<E, 64>(tS[m], 16 * w, 16 * i, lane);
            r1[m] = ld_row<E, 64>(tS[m], 16 * w, 16 * i + 16, lane);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            dB[nb] = mma_fb<E, 2>(ld_col<E, NT>(tC, 16 * i, 16 * nb, lane), ld_col<E, NT>(tC, 16 * i + 16, 16 * nb, lane), z0, z1, dB[nb]);
#pragma unroll
            for (int m = 0; m < NP; ++m)
                dC[nb] = mma(ld_col<E, NT>(tB, 16 * i, 16 * nb, lane), ld_col<E, NT>(tB, 16 * i + 16, 16 * nb, lane), r0[m], r1[m], dC[nb]);
        }
    }
    if (have) {
        float *o = gr.dbc + (((int64_t)hs * (gridDim.x / s.nchunk / gr.HS / s.G) + b) * s.L + t0 + mine) * 2 * s.G * s.N + g * s.N;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int n = 16 * nb + q4;
            if (n < s.N) {
                *reinterpret_cast<f32x4_t *>(o + n) = dB[nb];
                *reinterpret_cast<f32x4_t *>(o + s.G * s.N + n) = dC[nb];
            }
        }
    }
}

// dbc's HS parts of n elements each, added up in the first.
static __global__ void __launch_bounds__(256) sd_parts_kernel(float *dbc, int64_t n, int HS) {
    const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (e >= n) return;
    f32x4_t a = ld4(dbc + e);
#pragma unroll 8
    for (int i = 1; i < HS; ++i) a += ld4(dbc + i * n + e);
    *reinterpret_cast<f32x4_t *>(dbc + e) = a;
}

// Back through silu and the convolution; thread: kSdConvV channels of `tt` tokens, kSdConvT at a time, the next ones'
// rows requested before.  With g_t = du_t silu'(pre_t):
//   dx_t = sum_j w[j] g_{t+3-j},   dw[j] = sum g_t x_{t-3+j},   db = sum g_t         (w[j]: four taps, oldest first)
// so a thread forms g for three tokens past its own.  parts: [b * tile][5][dc] sums over the tile's tokens of dw's four
// taps and of db.
template <typename IO, bool AL>
__global__ void __launch_bounds__(256)
sd_conv_bwd_kernel(const IO *__restrict__ x, int64_t xstride, const float *__restrict__ w, const float *__restrict__ bias,
                   int width, const IO *__restrict__ st_in, const int32_t *__restrict__ lens, const float *__restrict__ du,
                   const float *__restrict__ dbc, IO *__restrict__ dx, IO *__restrict__ dst, float *__restrict__ parts,
                   int64_t L, int dc, int hp, int tt, int vblocks, int ntiles) {
    const int v = blockIdx.x % vblocks * 256 + threadIdx.x;
    if (v >= dc / kSdConvV) return;
    const int c = v * kSdConvV, bc = dc - hp;
    const int64_t b = blockIdx.x / vblocks / ntiles, tile = blockIdx.x / vblocks % ntiles, t0 = tile * tt, t1 = min(t0 + tt, L);
    const int64_t len = lens ? min(max((int64_t)lens[b], (int64_t)0), L) : L, end = min(t1 + 3, len);
    const IO *xb = x + b * L * xstride + c;
    const float *db_ = c < hp ? du + b * L * hp + c : dbc + b * L * bc + (c - hp);
    const int64_t drow = c < hp ? hp : bc;
    const int hw = width - 1;
    IO r[kSdConvT][kSdConvV] = {};
    f32x4_t d[kSdConvT] = {};
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < kSdConvT; ++i) {
            d[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            if (t + i < end) {
                conv_vec<IO, AL>::load(xb + (t + i) * xstride, r[i]);
                d[i] = ld4(db_ + (t + i) * drow);
            }
        }
    };
    fetch(t0);
    float wv[kSdTaps][kSdConvV], bv[kSdConvV], past[3][kSdConvV], g[kSdTaps][kSdConvV] = {}, aw[kSdTaps][kSdConvV] = {}, ab[kSdConvV] = {};
#pragma unroll
    for (int k = 0; k < kSdConvV; ++k) {
#pragma unroll
        for (int j = 0; j < kSdTaps; ++j) {
            const int tap = j - (kSdTaps - width);
            wv[j][k] = tap >= 0 ? w[(int64_t)(c + k) * width + tap] : 0.0f;
        }
        bv[k] = bias ? bias[c + k] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int64_t t = t0 - 3 + j;
        IO o[kSdConvV] = {};
        if (t >= 0) conv_vec<IO, AL>::load(xb + t * xstride, o);
        else if (st_in && t >= -hw) conv_vec<IO, true>::load(st_in + (b * hw + hw + t) * dc + c, o);
#pragma unroll
        for (int k = 0; k < kSdConvV; ++k) past[j][k] = io_f32(o[k]);
    }
    for (int64_t tb = t0; tb < t1 + 3; tb += kSdConvT) {
        IO rn[kSdConvT][kSdConvV];
        f32x4_t dn[kSdConvT];
#pragma unroll
        for (int i = 0; i < kSdConvT; ++i) {
            dn[i] = d[i];
#pragma unroll
            for (int k = 0; k < kSdConvV; ++k) rn[i][k] = r[i][k];
        }
        fetch(tb + kSdConvT);
#pragma unroll
        for (int i = 0; i < kSdConvT; ++i) {
            const int64_t t = tb + i;
            if (t >= t1 + 3) break;
            const bool live = t < len, own = t < t1;
#pragma unroll
            for (int k = 0; k < kSdConvV; ++k) {
                g[3][k] = g[2][k];   // g[j]: of token t - j
                g[2][k] = g[1][k];
                g[1][k] = g[0][k];
                const float now = io_f32(rn[i][k]);
                float p = fmaf(wv[0][k], past[0][k], bv[k]);
                p = fmaf(wv[1][k], past[1][k], p);
                p = fmaf(wv[2][k], past[2][k], p);
                p = fmaf(wv[3][k], now, p);
                const float sg = sigmoid_f32(p), gt = dn[i][k] * (sg * fmaf(p, 1.0f - sg, 1.0f));
                g[0][k] = live ? gt : 0.0f;   // (p may be NaN past the end)
                if (own && live) {
                    aw[0][k] = fmaf(gt, past[0][k], aw[0][k]);
                    aw[1][k] = fmaf(gt, past[1][k], aw[1][k]);
                    aw[2][k] = fmaf(gt, past[2][k], aw[2][k]);
                    aw[3][k] = fmaf(gt, now, aw[3][k]);
                    ab[k] += gt;
                }
                past[0][k] = past[1][k];
                past[1][k] = past[2][k];
                past[2][k] = now;
            }
            const int64_t to = t - 3;
            if (to >= t0 || (to < 0 && dst && to >= -hw)) {
                IO o[kSdConvV];
#pragma unroll
                for (int k = 0; k < kSdConvV; ++k) {
                    const float q = fmaf(wv[0][k], g[0][k], fmaf(wv[1][k], g[1][k], fmaf(wv[2][k], g[2][k], wv[3][k] * g[3][k])));
                    if constexpr (sizeof(IO) == 2) o[k] = f32_to_bf16(q);
                    else o[k] = q;
                }
                if (to >= 0) conv_vec<IO, true>::store(dx + (b * L + to) * dc + c, o);
                else conv_vec<IO, true>::store(dst + (b * hw + hw + to) * dc + c, o);
            }
        }
    }
    float *p = parts + (b * ntiles + tile) * 5 * dc + c;
#pragma unroll
    for (int j = 0; j < kSdTaps; ++j) *reinterpret_cast<f32x4_t *>(p + (int64_t)j * dc) = f32x4_t{aw[j][0], aw[j][1], aw[j][2], aw[j][3]};
    *reinterpret_cast<f32x4_t *>(p + 4 * (int64_t)dc) = f32x4_t{ab[0], ab[1], ab[2], ab[3]};
}

// Sums over n parts of `planes` planes of `cols` columns, in a fixed order, to the parameters' gradients:
// out[plane] + col * stride[plane] (null: not wanted).
struct sd_sums {
    float *out[5];
    int stride[5];
};
constexpr int kSdSumCols = 32, kSdSumGroups = 32;
static __global__ void __launch_bounds__(kSdSumCols *kSdSumGroups)
sd_sum_kernel(const float *__restrict__ part, int64_t n, int cols, int planes, sd_sums o) {
    __shared__ float red[kSdSumGroups][kSdSumCols + 1];
    const int col = threadIdx.x % kSdSumCols, g = threadIdx.x / kSdSumCols;
    const int cblocks = (cols + kSdSumCols - 1) / kSdSumCols, plane = blockIdx.x / cblocks;
    const int c = blockIdx.x % cblocks * kSdSumCols + col;
    float a = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t k = g; k < n; k += kSdSumGroups) a += part[(k * planes + plane) * cols + c];
    }
    red[g][col] = a;
    __syncthreads();
    if (g == 0 && c < cols && o.out[plane]) {
#pragma unroll
        for (int k = 1; k < kSdSumGroups; ++k) a += red[k][col];
        o.out[plane][(int64_t)c * o.stride[plane]] = a;
    }
}

}  // namespace ssm
