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
// FULL as in sd_scan_kernel.
// Bound: HBM where every chunk's state is written (B8 L2048 H80 N64 bf16, adjoints: 158 us, 506 MB, 3.2 TB/s), the chunks'
// chain otherwise (B1 L65536 H32 N128, 16 segments: 144 us).
template <typename E, int NT, bool ADJ, bool FULL>
__global__ void __launch_bounds__(kSdThreads)
sd_walk_kernel(const typename sd<E>::io *__restrict__ u_, const typename sd<E>::io *__restrict__ dy_,
               const float *__restrict__ tok, const int32_t *__restrict__ lens, const float *__restrict__ from, float *__restrict__ each,
               float *__restrict__ to, int ends, sd_shape s) {
    using IO = typename sd<E>::io;
    constexpr int NB = NT / 16;
    const int N = FULL ? NT : s.N;
    __shared__ __attribute__((aligned(16))) E tB[64 * sd_ld<E>(NT)], tX[64 * sd_ld<E>(64)];
    __shared__ sd_tokens tk;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const sd_segment at(s, lens);
    const int64_t b = at.b, len = at.len;
    const int h = at.h, pt = at.pt;
    const sd_view<IO> v(u_, s, b, h, pt);
    const int pw = FULL ? 64 : v.pw;
    const int xrow = ADJ ? s.H * s.P : s.dc;
    const E *xs = reinterpret_cast<const E *>(ADJ ? dy_ + (b * s.L * s.H + h) * s.P + pt * 64 : v.x);
    const E *Bs = reinterpret_cast<const E *>(ADJ ? v.C : v.B);
    tok += (b * s.H + h) * s.nchunk * kSdTok;
    f32x4_t S[NB];
    if (from) {
        sd_load_state(S, from + at.state_at(s, s.nseg, at.seg), N, pw, w, lane);
    } else {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    auto keep = [&](int64_t c) {
        if (each) sd_store_state(S, each + at.state_at(s, s.nchunk, c), N, pw, w, lane);
    };
    if (ADJ)   // chunks past the sequence's end leave the adjoint as it is
        for (int64_t c = at.live; c < at.c1; ++c) keep(c);
    tile64<E, NT> rB;
    tile64<E, 64> rX;
    sd_tok rt = {};
    auto fetch = [&](int64_t c) {
        const int64_t t0 = c * kSdQ;
        const int rows = (int)min((int64_t)64, len - t0);
        rB.load(Bs + t0 * s.dc, s.dc, rows, FULL ? NT : N);
        rX.load(xs + t0 * xrow, (uint32_t)xrow, rows, pw);
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
        for (int k = 0; k < 2; ++k) {
            const float *wt = (ADJ ? tk.e : tk.w) + 32 * k + 8 * (lane >> 4);
            const op32<E> x = col32<E, 64>(tX, 32 * k, 16 * w, lane);
            const formed<E> f0(widen(x.lo) * ld4(wt)), f1(widen(x.hi) * ld4(wt + 4));
#pragma unroll
            for (int n0 = 0; n0 < NB; n0 += 4) {
                op32<E> bv[4];
                f32x4_t add[4] = {};   // (the states on their accumulators, as in the scan, bit for bit)
#pragma unroll
                for (int nb = 0; nb < 4; ++nb) bv[nb] = col32<E, NT>(tB, 32 * k, 16 * (n0 + nb), lane);
#pragma unroll
                for (int m = 0; m < formed<E>::N; ++m)
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb) {
                        f32x4_t &to = ADJ ? add[nb] : S[n0 + nb];
                        to = mma(bv[nb].lo, bv[nb].hi, f0.p[m], f1.p[m], to);
                    }
                if (ADJ) {
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb) S[n0 + nb] += add[nb];
                }
            }
        }
        __syncthreads();
    }
    if (!ADJ)
        for (int64_t c = at.live; c < at.c1; ++c) keep(c);
    if (ends) sd_store_state(S, to + at.state_at(s, s.nseg, at.seg), N, pw, w, lane);
    else if (to && at.seg == (ADJ ? 0 : s.nseg - 1)) sd_store_state(S, to + at.state_at(s, 1, 0), N, pw, w, lane);
}

// What is formed in the backward is carried to 24 bits (three bf16 parts): the sums over tokens that u's gradient
// goes into leave in fp32.  For their sake too products that are not of a smaller part start from zero and are added up
// by vector instructions: the bf16 matrix instruction cuts its addend downward to 2^-24 of its largest product, a bias
// that sums over tokens collect (B8 L2048 H80 N64: the error of dt_bias's gradient 2.4e-6 that way).
constexpr int kSdBwdThreads = 1024;

// 64 x 64 of an adjoint [p][n] in fp32 from memory to LDS, as operand parts.
template <typename E> struct state64 {
    static constexpr int NP = formed<E>::N, NU = 1024 / kSdBwdThreads, RPP = kSdBwdThreads / 16;
    f32x4_t r[NU];
    __device__ __forceinline__ void load(const float *m, int N, int pw, int nw) {   // N: row stride; pw x nw exist
        const int p = threadIdx.x / 16, n = threadIdx.x % 16 * 4;
        const char *base = reinterpret_cast<const char *>(m);
        const uint32_t off = (uint32_t)(p * N + n) * 4u;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            r[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            if (p + RPP * i < pw && n < nw) r[i] = *reinterpret_cast<const f32x4_t *>(base + (int64_t)(RPP * i * N) * 4 + off);
        }
    }
    __device__ __forceinline__ void stage(E (&t)[NP][64 * sd_ld<E>(64)]) const {
        const int p = threadIdx.x / 16, n = threadIdx.x % 16 * 4;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            const formed<E> f(r[i]);
#pragma unroll
            for (int k = 0; k < NP; ++k) *reinterpret_cast<typename sd<E>::frag *>(&t[k][(p + RPP * i) * sd_ld<E>(64) + n]) = f.p[k];
        }
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

// One workgroup per (chunk, sequence, group, part of its heads), the heads in turn, the next one's rows and states
// requested while one is worked on.  Sixteen waves, four to a SIMD, of four kinds: kind 0 owns of every 64 states the
// 16 from 16 w of dC, kind 1 those of dB; kinds 2 and 3 (z = 0, 1) the 16 tokens 16 w .. of the chunk as s of T, G and v, of
// these the tokens t in blocks z and 3 - z of T and the channels 32 z .. of every 64 of v.
// MODE 1: whole tiles (P a multiple of 64, N = NT), without the checks for less; 2: and one item per head (P = N = 64).
// (MODE 2, 1 and 0: B8 L2048 H80 N64 bf16 347, 415 and 847 us, B2 L2048 H24 N64 fp32 68, 68 and 78; 1 and 0: B5 L777 H20
// N128 bf16 103 and 123.)
// The pairs of tokens are worked on once a head's 64 channels have their last states, 32 tokens t at a time: G, K, T and
// what comes of them then live for a few products only (351 us for B8 L2048 H80 N64 when this came, 492 with G K of all
// tokens held over a head).  Waves of kinds in loops of their own were taken as quicker than eight waves of every kind's work
// (559 there, before that) and four (683): a kind's accumulators stay in 128 registers.
// Bound: HBM, 1.5 GB in 347 us there (4.3 TB/s; each chunk's states and adjoints are 45 % of it), with vector
// instructions busy 56 % and LDS 39 % of the time beside it.
template <typename E, int NT, int MODE>
__global__ void __launch_bounds__(kSdBwdThreads) __attribute__((amdgpu_waves_per_eu(4)))
sd_bwd_kernel(const typename sd<E>::io *__restrict__ u_, const typename sd<E>::io *__restrict__ dy_,
              const float *__restrict__ tok, const typename sd<E>::io *__restrict__ dt, const float *__restrict__ A,
              const float *__restrict__ Dv, const float *__restrict__ dt_bias, const int32_t *__restrict__ lens,
              const float *__restrict__ st_in, const float *__restrict__ ds_out, typename sd<E>::io *__restrict__ ddt,
              sd_grad gr, sd_shape s) {
    using IO = typename sd<E>::io;
    using F = typename sd<E>::frag;
    constexpr bool FULL = MODE >= 1, ONE = MODE == 2;
    const int N = FULL ? NT : s.N, P = ONE ? 64 : s.P;
    constexpr int NH = NT / 64, NP = formed<E>::N, LD = sd_ld<E>(64);
    // Two sets of an item's tiles where they fit in LDS: the next item's are staged while one is worked on, and a
    // barrier an item is enough.
    constexpr int NBUF = sd<E>::split || NT == 64 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) E tB[64 * sd_ld<E>(NT)], tC[64 * sd_ld<E>(NT)], tXs[NBUF][64 * LD], tYs[NBUF][64 * LD];
    __shared__ __attribute__((aligned(16))) E tDs[NBUF][NP][64 * LD];
    // a head's tokens and sums (heads in turn)
    struct head_t {
        sd_tokens tk;
        float to_end[64], near[64], sig[64];            // e^{c_last - c_t}; e^{c_t - c_r}, r the first of t's 16 tokens; softplus'
        float R[4][64], YS[4][64], col[2][64], XS[2][64], Q[2][64], XY[2][64], dot[4];
    };
    __shared__ __attribute__((aligned(16))) head_t hd[2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kind = wave >> 2, z = kind & 1;
    // (a SIMD's waves are those of one wave % 4; the tokens' blocks have less to do the later they are)
    const int w = kind == 3 ? 3 - (wave & 3) : wave & 3;
    const bool first = wave < kSdBwdThreads / 128;   // this half of the threads moves B and x, the other C and dy
    const int tid = threadIdx.x % (kSdBwdThreads / 2);
    const int c16 = lane & 15, q4 = 4 * (lane >> 4), mine = 16 * w + c16;   // mine: the lane's token of the wave's 16
    const uint32_t nchunk = (uint32_t)s.nchunk, chunk = blockIdx.x % nchunk, rest = blockIdx.x / nchunk;
    const int hs = rest % (uint32_t)gr.HS, g = rest / (uint32_t)gr.HS % (uint32_t)s.G;
    const uint32_t b = rest / (uint32_t)gr.HS / (uint32_t)s.G;
    const int64_t t0 = (int64_t)chunk * kSdQ;
    const int per = s.H / s.G, h0 = g * per + hs * gr.hpw, h1 = min(h0 + gr.hpw, (g + 1) * per);
    const int64_t len = lens ? min(max((int64_t)lens[b], (int64_t)0), s.L) : s.L;
    const int rows = (int)min((int64_t)64, max(len - t0, (int64_t)0)), tokens = (int)min((int64_t)64, s.L - t0);
    const bool have = mine < tokens;
    const IO *ub = u_ + (b * s.L + t0) * s.dc, *dyb = dy_ + (b * s.L + t0) * s.H * P;

    // An item: 64 states of 64 channels of a head.
    struct item_t {
        int h, pt, nh;
    };
    auto next = [&](item_t i) -> item_t {
        if (ONE) return {i.h + 1, 0, 0};
        if (i.nh + 64 < N) return {i.h, i.pt, i.nh + 64};
        if (i.pt + 1 < (P + 63) / 64) return {i.h, i.pt + 1, 0};
        return {i.h + 1, 0, 0};
    };
    tile64<E, 64, kSdBwdThreads / 2> rXY;
    state64<E> rD;
    f32x4_t rS[4];                       // (kind 0) the state entering, as operand: rows n (this wave's 16), k = p
    auto state_at = [&](item_t i) {
        return ((int64_t)((b * s.H + i.h) * nchunk + chunk) * P + (int64_t)i.pt * 64) * N + i.nh;
    };
    auto fetch = [&](item_t i) {         // the tiles
        if (i.h >= h1) return;
        const int pw = FULL ? 64 : min(64, P - i.pt * 64);
        if (i.nh == 0) {
            rXY.load(reinterpret_cast<const E *>((first ? ub : dyb) + i.h * P + i.pt * 64), (uint32_t)(first ? s.dc : s.H * P), rows, pw, tid);
        }
        rD.load(ds_out + state_at(i), N, pw, FULL ? 64 : N - i.nh);
    };
    auto fetch_state = [&](item_t i) {
        if (i.h >= h1 || kind != 0) return;
        const int pw = FULL ? 64 : min(64, P - i.pt * 64);
        const char *m = reinterpret_cast<const char *>(st_in + state_at(i));
        const uint32_t off = (uint32_t)(2 * q4 * N + mine) * 4u, row = (uint32_t)N * 4u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {   // channels 32 (k / 2) + 8 (lane / 16) + 4 (k % 2) .. + 3, which exist or not as a whole
            const int p0 = 32 * (k >> 1) + 4 * (k & 1);
            rS[k] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            if (FULL || (p0 + 2 * q4 < pw && mine < N - i.nh)) {
                const uint32_t at = off + p0 * row;
#pragma unroll
                for (int e = 0; e < 4; ++e) rS[k][e] = *reinterpret_cast<const float *>(m + (size_t)(e * row) + at);
            }
        }
    };
    int xbuf = 0, dbuf = 0;              // the current item's buffers (x and dy are a head's 64 channels', dS an item's)
    auto stage = [&](item_t i, int xb, int db) {
        if (i.h >= h1) return;
        if (i.nh == 0) {
            rXY.stage(first ? tXs[xb] : tYs[xb], tid);
        }
        rD.stage(tDs[db]);
    };
    // One wave's (of kind 1, the last): the next head's tokens, token = lane.
    sd_tok rt = {};
    float rraw = 0.0f;
    auto fetch_tokens = [&](int h) {
        if (h >= h1) return;
        rt = sd_load_tokens(tok + (int64_t)((b * s.H + h) * nchunk + chunk) * kSdTok, lane);
        if (lane < rows) rraw = io<IO>::ld(dt, ((int64_t)b * s.L + t0 + lane) * s.dt_stride + h) + (dt_bias ? dt_bias[h] : 0.0f);
    };
    auto stage_tokens = [&](int h) {
        if (h >= h1) return;
        head_t &n = hd[h & 1];
        n.to_end[lane] = sd_stage_tokens(n.tk, rt, lane);
        const float rh = __shfl(rt.h, lane & 48, 64), rl = __shfl(rt.l, lane & 48, 64);
        n.near[lane] = hw_exp2((rt.h - rh) + (rt.l - rl));
        float sig = 1.0f;
        if (s.softplus) softplus_f32(rraw, sig);
        n.sig[lane] = lane < rows ? sig : 0.0f;
    };
    // and from a head's sums over pairs of tokens to its gradients
    auto finish = [&](int h) {
        head_t &n = hd[h & 1];
        const float a = A[h];
        const double v = (double)(n.R[0][lane] + n.R[1][lane] + n.R[2][lane] + n.R[3][lane]) - (n.col[0][lane] + n.col[1][lane]) +
                         (n.YS[0][lane] + n.YS[1][lane] + n.YS[2][lane] + n.YS[3][lane]);
        const double p = wave_incl_sum64(v), x = n.XS[0][lane] + n.XS[1][lane], px = wave_incl_sum64(x);
        const double ends = (double)n.tk.dec * ((n.dot[0] + n.dot[1]) + (n.dot[2] + n.dot[3]));
        const float dg = (float)((wave_last(p) - p + v) + (px - x) + ends);
        const float dr = (n.Q[0][lane] + n.Q[1][lane] + a * dg) * n.sig[lane];
        if (lane < tokens) io<IO>::st(ddt, (b * s.L + t0 + lane) * s.H + h, dr);
        const float pa = wave_sum(n.tk.dt[lane] * dg), pb = wave_sum(dr), pd = wave_sum(n.XY[0][lane] + n.XY[1][lane]);
        if (lane == 0) {
            float *o = gr.part + (b * s.nchunk + chunk) * 3 * s.H + h;
            o[0] = pa;
            o[s.H] = pb;
            o[2 * s.H] = pd;
        }
    };
    // The kinds' loops over the items are apart, so that each kind's registers are its own; every wave comes by the
    // same barriers: one (two with a single set of tiles) at an item's start, two at the end.
    const item_t start = {h0, 0, 0};
    {
        tile64<E, NT, kSdBwdThreads / 2> rBC;
        rBC.load(reinterpret_cast<const E *>(ub + s.H * P + g * N) + (first ? 0 : s.G * N), (uint32_t)s.dc, rows, FULL ? NT : N, tid);
        fetch(start);
        rBC.stage(first ? tB : tC, tid);
        if constexpr (NBUF == 2) {
            stage(start, 0, 0);
            fetch(next(start));
        }
        if (wave == 7) {
            fetch_tokens(h0);
            stage_tokens(h0);
            fetch_tokens(h0 + 1);
        }
    }
    auto begin = [&](item_t now, item_t then) {
        __syncthreads();
        if constexpr (NBUF == 2) {
            stage(then, xbuf ^ (then.nh == 0), dbuf ^ 1);
            fetch(next(then));
        } else {
            stage(now, 0, 0);
            fetch(then);
            __syncthreads();
        }
    };
    auto turn = [&](item_t then) {   // to the other buffers
        if constexpr (NBUF == 2) {
            xbuf ^= then.nh == 0;
            dbuf ^= 1;
        }
    };
    using parts_t = E[NP][64 * LD];
    // kinds 0 and 1, in the end: the products that the group's heads share, with Z [t][s] in LDS.  src: C for dB (over
    // t), B for dC (over s)
    auto shared_products = [&](f32x4_t (&acc)[NH][4], const E *src, bool over_t) {
        const parts_t &tZ = tDs[0];
        float *o = gr.dbc + (((int64_t)hs * (gridDim.x / nchunk / (uint32_t)gr.HS / (uint32_t)s.G) + b) * s.L + t0) * 2 * s.G * N + g * N + (over_t ? 0 : s.G * N);
#pragma unroll
        for (int half = 0; half < NH; ++half) {
            const int n0 = 64 * half + 16 * w;
            if (64 * half >= N) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const op32<E> f = col32<E, NT>(src, 32 * i, n0, lane);
                f32x4_t add[4] = {};
#pragma unroll
                for (int m = 0; m < NP; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        add[j] = mma(f, over_t ? col32<E, 64>(tZ[m], 32 * i, 16 * j, lane) : row32<E, 64>(tZ[m], 16 * j, 32 * i, lane), add[j]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[half][j] += add[j];
            }
            if (FULL || n0 + q4 < N) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (16 * j + c16 < tokens) *reinterpret_cast<f32x4_t *>(o + (int64_t)(16 * j + c16) * 2 * s.G * N + n0 + q4) = acc[half][j];
            }
        }
    };
    if (kind == 0) {   // through the state entering: dC^T[n][t]
        // (two blocks of tokens at a time where both halves' accumulators are held: with four they spill, B5 L777 H20 N128
        // 117 us for 103; with two at N <= 64 the B8 case takes 509 for 347, B2 L2048 H24 fp32 65 for 68)
        constexpr int kTogether = NH == 1 ? 4 : 2;
        f32x4_t acc[NH][4] = {};
        float dot = 0.0f, ys[4] = {};
        fetch_state(start);
        for (item_t now = start, then = next(now); now.h < h1; now = then, then = next(then)) {
            begin(now, then);
            const sd_tokens &tk = hd[now.h & 1].tk;
            const E *tY = tYs[xbuf];
            const parts_t &tD = tDs[dbuf];
            const formed<E> S[4] = {formed<E>(rS[0]), formed<E>(rS[1]), formed<E>(rS[2]), formed<E>(rS[3])};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                op32<E> d = col32<E, 64>(tD[0], 32 * k, 16 * w, lane);
                f32x4_t lo = widen(d.lo), hi = widen(d.hi);
#pragma unroll
                for (int m = 1; m < NP; ++m) {
                    d = col32<E, 64>(tD[m], 32 * k, 16 * w, lane);
                    lo += widen(d.lo);
                    hi += widen(d.hi);
                }
                lo = lo * rS[2 * k] + hi * rS[2 * k + 1];
                dot += (lo[0] + lo[1]) + (lo[2] + lo[3]);
            }
            fetch_state(then);
#pragma unroll
            for (int half = 0; half < NH; ++half) {
                if (now.nh != 64 * half) continue;
#pragma unroll kTogether
                for (int j = 0; j < 4; ++j) {
                    const op32<E> y0 = row32<E, 64>(tY, 16 * j, 0, lane), y1 = row32<E, 64>(tY, 16 * j, 32, lane);
                    f32x4_t c0 = {}, c1 = {};
#pragma unroll
                    for (int m = 0; m < NP; ++m) {
                        c0 = mma(S[0].p[m], S[1].p[m], y0.lo, y0.hi, c0);
                        c1 = mma(S[2].p[m], S[3].p[m], y1.lo, y1.hi, c1);
                    }
                    c0 = (c0 + c1) * tk.e[16 * j + c16];
                    const f32x4_t cf = widen(ld_row<E, NT>(tC, 16 * j, 64 * half + 16 * w, lane));
                    acc[half][j] += c0;
                    ys[j] += c0[0] * cf[0] + c0[1] * cf[1] + c0[2] * cf[2] + c0[3] * cf[3];
                }
            }
            if (then.h != now.h) {
                head_t &hn = hd[now.h & 1];
                dot = wave_sum(dot);
                if (lane == 0) hn.dot[w] = dot;
                dot = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float r = quads_sum(ys[j]);
                    if (lane < 16) hn.YS[w][16 * j + c16] = r;
                    ys[j] = 0.0f;
                }
            }
            turn(then);
        }
        __syncthreads();
        __syncthreads();
        shared_products(acc, tB, false);
    } else if (kind == 1) {   // through the state leaving: dB^T[n][s]
        f32x4_t acc[NH][4] = {};
        for (item_t now = start, then = next(now); now.h < h1; now = then, then = next(then)) {
            begin(now, then);
            if (wave == 7 && now.nh == 0 && now.pt == 0) {   // (the head before is done, its tokens' place free)
                if (now.h > h0) finish(now.h - 1);
                stage_tokens(now.h + 1);
                fetch_tokens(now.h + 2);
            }
            const sd_tokens &tk = hd[now.h & 1].tk;
            const E *tX = tXs[xbuf];
            const parts_t &tD = tDs[dbuf];
            op32<E> d0[NP][2];
#pragma unroll
            for (int m = 0; m < NP; ++m)
#pragma unroll
                for (int k = 0; k < 2; ++k) d0[m][k] = col32<E, 64>(tD[m], 32 * k, 16 * w, lane);
#pragma unroll
            for (int half = 0; half < NH; ++half) {
                if (now.nh != 64 * half) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const op32<E> x0 = row32<E, 64>(tX, 16 * j, 0, lane), x1 = row32<E, 64>(tX, 16 * j, 32, lane);
                    f32x4_t c0 = {}, c1 = {};
#pragma unroll
                    for (int m = 0; m < NP; ++m) {
                        c0 = mma(d0[m][0], x0, c0);
                        c1 = mma(d0[m][1], x1, c1);
                    }
                    acc[half][j] += (c0 + c1) * tk.w[16 * j + c16];
                }
            }
            turn(then);
        }
        __syncthreads();
        if (wave == 7) finish(h1 - 1);
        __syncthreads();
        shared_products(acc, tC, true);
    } else {
        // blocks of tokens t: z and 3 - z, of which those before w have nothing
        const int tb[2] = {z, 3 - z};
        f32x4_t Z[2] = {}, V[2];
        float xs = 0.0f, q = 0.0f, xy = 0.0f, col = 0.0f;
        for (item_t now = start, then = next(now); now.h < h1; now = then, then = next(then)) {
            begin(now, then);
            head_t &hn = hd[now.h & 1];
            const sd_tokens &tk = hn.tk;
            const E *tX = tXs[xbuf], *tY = tYs[xbuf];
            const parts_t &tD = tDs[dbuf];
            if (now.nh == 0) V[0] = V[1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            // through the state leaving: V^T[p][s]
#pragma unroll
            for (int k = 0; k < 64; k += 32) {
                const op32<E> bv = row32<E, NT>(tB, 16 * w, now.nh + k, lane);
                f32x4_t add[2] = {};
#pragma unroll
                for (int m = 0; m < NP; ++m)
#pragma unroll
                    for (int j = 0; j < 2; ++j) add[j] = mma(row32<E, 64>(tD[m], 32 * z + 16 * j, k, lane), bv, add[j]);
                V[0] += add[0];
                V[1] += add[1];
            }
            if (then.nh == 0) {   // the 64 channels' last states: the pairs of tokens (all linear in the channels)
                const int pw = FULL ? 64 : min(64, P - now.pt * 64);
                const float te = hn.to_end[mine], d = tk.dt[mine], sh = tk.ch[mine], sl = tk.cl[mine];
                f32x4_t x[2];
                float x0 = 0.0f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    V[j] *= te;
                    x[j] = widen(ld_row<E, 64>(tX, 16 * w, 32 * z + 16 * j, lane));
                    x0 += V[j][0] * x[j][0] + V[j][1] * x[j][1] + V[j][2] * x[j][2] + V[j][3] * x[j][3];
                }
                xs += x0 * d;
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const int mineb = tb[i / 2], t = 16 * mineb + q4;   // the pair's block whose T is the wave's
                    if (mineb < w && c16 < 4 && now.pt == 0) hn.R[w][t + c16] = 0.0f;
                    if (i + 1 < w) continue;
                    f32x4_t gk[2], kk[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        gk[u] = kk[u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
                        if (i + u < w) continue;
                        f32x4_t G = {};
#pragma unroll
                        for (int k = 0; k < NT; k += 32) G += mma(row32<E, NT>(tC, 16 * (i + u), k, lane), row32<E, NT>(tB, 16 * w, k, lane), f32x4_t{});
                        if (i + u == w) {
                            const f32x4_t th = ld4(tk.ch + 16 * (i + u) + q4), tl = ld4(tk.cl + 16 * (i + u) + q4);
#pragma unroll
                            for (int e = 0; e < 4; ++e) kk[u][e] = q4 + e >= c16 ? hw_exp2((th[e] - sh) + (tl[e] - sl)) : 0.0f;
                        } else {   // in two factors of at most 1, over the block's first token
                            kk[u] = ld4(hn.near + 16 * (i + u) + q4) * hw_exp2((tk.ch[16 * (i + u)] - sh) + (tk.cl[16 * (i + u)] - sl));
                        }
                        gk[u] = G * kk[u];
                    }
                    if (mineb >= w) {
                        f32x4_t T = {};
#pragma unroll
                        for (int k = 0; k < 64; k += 32) T += mma(row32<E, 64>(tY, 16 * mineb, k, lane), row32<E, 64>(tX, 16 * w, k, lane), f32x4_t{});
                        T *= d;
                        const bool second = mineb != i;   // (the wave's: a copy by selection)
                        Z[i / 2] += T * (second ? kk[1] : kk[0]);
                        T *= second ? gk[1] : gk[0];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float wv = t + e > mine ? T[e] : 0.0f;
                            col += wv;
                            const float r = lanes_sum<16>(wv);
                            if (c16 == 0) hn.R[w][t + e] = ONE || now.pt == 0 ? r : hn.R[w][t + e] + r;
                        }
                    }
                    const formed<E> g0(gk[0]), g1(gk[1]);
                    F y0[2], y1[2];
                    f32x4_t add[2] = {};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        y0[j] = ld_col<E, 64>(tY, 16 * i, 32 * z + 16 * j, lane);
                        y1[j] = ld_col<E, 64>(tY, 16 * i + 16, 32 * z + 16 * j, lane);
                    }
#pragma unroll
                    for (int m = 0; m < NP; ++m)
#pragma unroll
                        for (int j = 0; j < 2; ++j) add[j] = mma(y0[j], y1[j], g0.p[m], g1.p[m], add[j]);
                    V[0] += add[0];
                    V[1] += add[1];
                }
                const float skip = Dv ? Dv[now.h] : 0.0f;
                char *o = reinterpret_cast<char *>(gr.du + ((b * s.L + t0) * s.H + now.h) * P + now.pt * 64);
                const uint32_t off = ((uint32_t)mine * (uint32_t)(s.H * P) + (uint32_t)(32 * z + q4)) * 4u;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const f32x4_t y = widen(ld_row<E, 64>(tY, 16 * w, 32 * z + 16 * j, lane));
                    q += V[j][0] * x[j][0] + V[j][1] * x[j][1] + V[j][2] * x[j][2] + V[j][3] * x[j][3];
                    xy += x[j][0] * y[0] + x[j][1] * y[1] + x[j][2] * y[2] + x[j][3] * y[3];
                    if (have && (FULL || 32 * z + 16 * j + q4 < pw)) *reinterpret_cast<f32x4_t *>(o + (off + 64 * j)) = V[j] * d + y * skip;
                }
            }
            if (then.h != now.h) {   // the head's sums over the tokens
                col = quads_sum(col);
                xs = quads_sum(xs);
                q = quads_sum(q);
                xy = quads_sum(xy);
                if (lane < 16) {
                    hn.col[z][mine] = col;
                    hn.XS[z][mine] = xs;
                    hn.Q[z][mine] = q;
                    hn.XY[z][mine] = xy;
                }
                xs = q = xy = col = 0.0f;
            }
            turn(then);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const formed<E> f(Z[j]);
#pragma unroll
            for (int m = 0; m < NP; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) tDs[0][m][(16 * tb[j] + q4 + e) * LD + mine] = f.p[m][e];
        }
        __syncthreads();
    }
}

// dbc's HS parts of n elements each, added up in the first (HBM; 4.8 us for B2 L2048 G1 N64).
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
// so a thread forms g for three tokens past its own.  W4 as in sd_conv_kernel (a tap that is not there takes no g
// either).  Bound: HBM (B8 L2048 of 5,248 channels bf16: 149 us, 688 MB, 4.6 TB/s; B2 L2048 of 1,664 fp32 20 us).
// parts: [b * tile][5][dc] sums over the tile's tokens of dw's four taps and of db.
template <typename IO, bool AL, bool W4>
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
    conv_weights(w, width, c, wv);
    conv_bias(bias, c, bv);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int64_t t = t0 - 3 + j;
        IO o[kSdConvV] = {};
        if (t >= 0) conv_vec<IO, AL>::load(xb + t * xstride, o);
        else if (st_in && t >= -hw) conv_vec<IO, true>::load(st_in + (b * hw + hw + t) * dc + c, o);
#pragma unroll
        for (int k = 0; k < kSdConvV; ++k) past[j][k] = W4 || hw >= 3 - j ? io_f32(o[k]) : 0.0f;
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
                past[0][k] = W4 || hw >= 3 ? past[1][k] : 0.0f;
                past[1][k] = W4 || hw >= 2 ? past[2][k] : 0.0f;
                past[2][k] = W4 || hw >= 1 ? now : 0.0f;
            }
            const int64_t to = t - 3;
            if (to >= t0 || (to < 0 && dst && to >= -hw)) {
                IO o[kSdConvV];
#pragma unroll
                for (int k = 0; k < kSdConvV; ++k) {
                    const float g0 = W4 || hw >= 3 ? g[0][k] : 0.0f, g1 = W4 || hw >= 2 ? g[1][k] : 0.0f, g2 = W4 || hw >= 1 ? g[2][k] : 0.0f;
                    const float q = fmaf(wv[0][k], g0, fmaf(wv[1][k], g1, fmaf(wv[2][k], g2, wv[3][k] * g[3][k])));
                    if constexpr (sizeof(IO) == 2) o[k] = f32_to_bf16(q);
                    else o[k] = q;
                }
                if (to >= 0) conv_store<IO>(dx + (b * L + to) * dc + c, o);
                else conv_store<IO>(dst + (b * hw + hw + to) * dc + c, o);
            }
        }
    }
    float *p = parts + (b * ntiles + tile) * 5 * dc + c;
#pragma unroll
    for (int j = 0; j < kSdTaps; ++j) *reinterpret_cast<f32x4_t *>(p + (int64_t)j * dc) = f32x4_t{aw[j][0], aw[j][1], aw[j][2], aw[j][3]};
    *reinterpret_cast<f32x4_t *>(p + 4 * (int64_t)dc) = f32x4_t{ab[0], ab[1], ab[2], ab[3]};
}

// Sums over n parts of `planes` planes of `cols` columns, in a fixed order and in 64 bits (the parts cancel), to the parameters' gradients:
// out[plane] + col * stride[plane] (null: not wanted).
struct sd_sums {
    float *out[5];
    int stride[5];
};
constexpr int kSdSumCols = 32, kSdSumGroups = 32;
static __global__ void __launch_bounds__(kSdSumCols *kSdSumGroups)
sd_sum_kernel(const float *__restrict__ part, int64_t n, int cols, int planes, sd_sums o) {
    __shared__ double red[kSdSumGroups][kSdSumCols + 1];
    const int col = threadIdx.x % kSdSumCols, g = threadIdx.x / kSdSumCols;
    const int cblocks = (cols + kSdSumCols - 1) / kSdSumCols, plane = blockIdx.x / cblocks;
    const int c = blockIdx.x % cblocks * kSdSumCols + col;
    double a = 0.0;
    if (c < cols) {
#pragma unroll 8
        for (int64_t k = g; k < n; k += kSdSumGroups) a += part[(k * planes + plane) * cols + c];
    }
    red[g][col] = a;
    __syncthreads();
    if (g == 0 && c < cols && o.out[plane]) {
#pragma unroll
        for (int k = 1; k < kSdSumGroups; ++k) a += red[k][col];
        o.out[plane][(int64_t)c * o.stride[plane]] = (float)a;
    }
}

}  // namespace ssm
