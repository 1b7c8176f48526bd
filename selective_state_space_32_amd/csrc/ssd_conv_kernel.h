// The state space dual layer with its short convolution: prompts, single tokens, gradients.
//
// Per head h (P channels, its group's B and C of N states), with u = silu(conv) rounded to the I/O
// type, dt = softplus(raw + bias) and g = A dt the logarithm of a token's decay:
//   S_t = e^{g_t} S_{t-1} + dt_t x_t B_t^T,   y_t = S_t C_t + D x_t
// Over a chunk of 64 tokens, with c_t = g_0 + .. + g_t, K[t,s] = e^{c_t - c_s} for s <= t, and S the
// state entering the chunk:
//   G = C B^T,  M[t,s] = G[t,s] K[t,s] dt_s,   Y = M X + e^{c_t} C S^T + D X
//   S <- e^{c_last} S + sum_s (e^{c_last - c_s} dt_s x_s) B_s^T
#pragma once

#include <type_traits>

#include "device_math.h"

namespace ssm {

constexpr int kSdQ = 64;           // tokens per chunk
constexpr int kSdThreads = 256;    // four waves; wave w owns the 16 channels 16 w .. of a 64-channel tile
constexpr int kSdTaps = 4;         // taps of the convolution at most
constexpr int kSdConvV = 4;        // channels per thread of the convolution's kernels
constexpr int kSdParts = 3;        // bf16 parts of an operand that is formed in fp32

// ---- operands of the matrix products --------------------------------------------------------
//
// An operand comes in fragments of 16 values of the contraction index k: lane l holds, for its row
// (A) or column (B) l % 16, the four consecutive k at 4 (l / 16).  That is also the layout of an
// accumulator (rows 4 (l / 16) + e, column l % 16), so an accumulator is a fragment of the product
// that contracts over its rows without leaving its registers.  bf16: two fragments make one operand of
// v_mfma_f32_16x16x32_bf16 (both operands order k alike); fp32: a fragment feeds four
// v_mfma_f32_16x16x4_f32.  Operands that are formed in fp32 are split into three bf16 parts of 8 bits each, which hold
// fp32's 24.  (Two, 16 bits, took 263 us in place of 282 for prompts of B8 L2048 H80 N64 and 766 in place of 826 for B1 L65536
// H32 N128, but left bf16 outputs 1.1e-4 of their root mean square from the roundings of fp32's; now 1.1e-5 to 2.7e-5.)
typedef __bf16 sd_bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 sd_bf16x8 __attribute__((ext_vector_type(8)));
typedef short sd_i16x4 __attribute__((ext_vector_type(4)));

template <typename E> struct sd;
template <> struct sd<__bf16> {
    using io = uint16_t;
    using frag = sd_bf16x4;
    static constexpr int pad = 8;
    static constexpr bool split = true;
};
template <> struct sd<float> {
    using io = float;
    using frag = f32x4_t;
    static constexpr int pad = 4;
    static constexpr bool split = false;
};
// Row stride of a tile of W columns in LDS: rows start 16 bytes apart modulo the banks.
template <typename E> constexpr int sd_ld(int w) { return w + sd<E>::pad; }

// k contiguous in the tile: four values of row r0 + l % 16 from column k0 + 4 (l / 16)
template <typename E, int W>
__device__ __forceinline__ typename sd<E>::frag ld_row(const E *t, int r0, int k0, int lane) {
    return *reinterpret_cast<const typename sd<E>::frag *>(t + (r0 + (lane & 15)) * sd_ld<E>(W) + k0 + 4 * (lane >> 4));
}
// k along the tile's rows: column m0 + l % 16 of rows k0 + 4 (l / 16) .. + 3.  (bf16: the transposing LDS
// read returns to lane j of a group of 16 the four rows' element j % 16 of the 4 x 16 block that the
// group addresses, lane i row i / 4, columns 4 (i % 4).)
template <typename E, int W>
__device__ __forceinline__ typename sd<E>::frag ld_col(const E *t, int k0, int m0, int lane) {
    if constexpr (sd<E>::split) {
        const int i = lane & 15;
        typedef __attribute__((address_space(3))) sd_i16x4 lds_i16x4;
        const __bf16 *p = t + (k0 + 4 * (lane >> 4) + (i >> 2)) * sd_ld<E>(W) + m0 + 4 * (i & 3);
        return __builtin_bit_cast(sd_bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)p));
    } else {
        const float *p = t + (k0 + 4 * (lane >> 4)) * sd_ld<E>(W) + m0 + (lane & 15);
        return f32x4_t{p[0], p[sd_ld<E>(W)], p[2 * sd_ld<E>(W)], p[3 * sd_ld<E>(W)]};
    }
}
__device__ __forceinline__ f32x4_t mma(sd_bf16x4 a0, sd_bf16x4 a1, sd_bf16x4 b0, sd_bf16x4 b1, f32x4_t c) {
    const sd_bf16x8 a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
    const sd_bf16x8 b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma(f32x4_t a0, f32x4_t a1, f32x4_t b0, f32x4_t b1, f32x4_t c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a0[e], b0[e], c, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a1[e], b1[e], c, 0, 0, 0);
    return c;
}
// A fragment formed in fp32, in parts (one with fp32 operands).
template <typename E> struct formed {
    static constexpr int N = sd<E>::split ? kSdParts : 1;
    typename sd<E>::frag p[N];
    __device__ __forceinline__ formed() {}
    __device__ __forceinline__ explicit formed(f32x4_t v) {
        if constexpr (sd<E>::split) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __bf16 h = (__bf16)v[e];
                    p[i][e] = h;
                    if (i + 1 < N) v[e] -= (float)h;
                }
        } else {
            p[0] = v;
        }
    }
};
// Two fragments of operands that both come from LDS, whose order of k is free: a lane holds the eight consecutive k at
// 8 (l / 16) of a 32-wide step (16-byte reads move twice the bytes of 8-byte ones in the same time).
template <typename E> struct op32 {
    typename sd<E>::frag lo, hi;
};
template <typename E, int W> __device__ __forceinline__ op32<E> row32(const E *t, int r0, int k0, int lane) {
    const E *p = t + (r0 + (lane & 15)) * sd_ld<E>(W) + k0 + 8 * (lane >> 4);
    if constexpr (sd<E>::split) {
        const sd_bf16x8 v = *reinterpret_cast<const sd_bf16x8 *>(p);
        return {__builtin_shufflevector(v, v, 0, 1, 2, 3), __builtin_shufflevector(v, v, 4, 5, 6, 7)};
    } else {
        return {*reinterpret_cast<const f32x4_t *>(p), *reinterpret_cast<const f32x4_t *>(p + 4)};
    }
}
template <typename E, int W> __device__ __forceinline__ op32<E> col32(const E *t, int k0, int m0, int lane) {
    if constexpr (sd<E>::split) {
        const int i = lane & 15;
        typedef __attribute__((address_space(3))) sd_i16x4 lds_i16x4;
        const __bf16 *p = t + (k0 + 8 * (lane >> 4) + (i >> 2)) * sd_ld<E>(W) + m0 + 4 * (i & 3);
        return {__builtin_bit_cast(sd_bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)p)),
                __builtin_bit_cast(sd_bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(p + 4 * sd_ld<E>(W))))};
    } else {
        constexpr int LD = sd_ld<E>(W);
        const float *p = t + (k0 + 8 * (lane >> 4)) * LD + m0 + (lane & 15);
        return {f32x4_t{p[0], p[LD], p[2 * LD], p[3 * LD]}, f32x4_t{p[4 * LD], p[5 * LD], p[6 * LD], p[7 * LD]}};
    }
}
template <typename E> __device__ __forceinline__ f32x4_t mma(const op32<E> &a, const op32<E> &b, f32x4_t c) {
    return mma(a.lo, a.hi, b.lo, b.hi, c);
}
__device__ __forceinline__ f32x4_t widen(sd_bf16x4 v) { return f32x4_t{(float)v[0], (float)v[1], (float)v[2], (float)v[3]}; }
__device__ __forceinline__ f32x4_t widen(f32x4_t v) { return v; }

// ---- tiles ----------------------------------------------------------------------------------

// 64 rows (tokens) of W elements between memory and LDS, 16 bytes per thread and access.  Addresses are a
// uniform base and a 32-bit offset per lane (64 rows of at most 2^23 elements of 4 bytes).
template <typename E, int W, int THREADS = kSdThreads> struct tile64 {
    static constexpr int EPU = 16 / (int)sizeof(E);           // elements per unit
    static constexpr int UPR = W / EPU;                       // units per row
    static constexpr int NU = 64 * UPR / THREADS;             // units per thread
    static constexpr int RPP = THREADS / UPR;                 // rows per pass
    static_assert(64 * UPR % THREADS == 0, "whole units per thread");
    u32x4_t r[NU];
    // rows [0, rows) of `src` (elements `stride` apart), columns [0, cols); zeros elsewhere
    __device__ __forceinline__ void load(const E *src, uint32_t stride, int rows, int cols, int tid = threadIdx.x) {
        const int row = tid / UPR, c = tid % UPR * EPU;
        const uint32_t off = ((uint32_t)row * stride + (uint32_t)c) * (uint32_t)sizeof(E), step = RPP * stride * (uint32_t)sizeof(E);
        const char *base = reinterpret_cast<const char *>(src);
        if (rows >= 64 && cols >= W) {
#pragma unroll
            for (int i = 0; i < NU; ++i) r[i] = *reinterpret_cast<const u32x4_t *>(base + (off + i * step));
        } else {
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                r[i] = u32x4_t{0u, 0u, 0u, 0u};
                if (row + RPP * i < rows && c < cols) r[i] = *reinterpret_cast<const u32x4_t *>(base + (off + i * step));
            }
        }
    }
    __device__ __forceinline__ void stage(E *t, int tid = threadIdx.x) const {
        const int row = tid / UPR, c = tid % UPR * EPU;
#pragma unroll
        for (int i = 0; i < NU; ++i) *reinterpret_cast<u32x4_t *>(t + (row + RPP * i) * sd_ld<E>(W) + c) = r[i];
    }
};

// Inclusive sum over the 64 lanes of a wave in 64 bits: the logarithms of a chunk's decays add up to
// hundreds, and their differences are exponents.
__device__ __forceinline__ double wave_incl_sum64(double v) {
    auto moved = [](double x, auto ctrl, auto mask) {
        const uint64_t b = __builtin_bit_cast(uint64_t, x);
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, ctrl.value, mask.value, 0xf, false);
        const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), ctrl.value, mask.value, 0xf, false);
        return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    };
    using std::integral_constant;
    v += moved(v, integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});   // row_shr 1, 2, 4, 8
    v += moved(v, integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
    v += moved(v, integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
    v += moved(v, integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
    v += moved(v, integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});   // row_bcast 15, 31
    v += moved(v, integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});
    return v;
}
// A chunk's per-token values.  c_t = log2 e^{g_0 + .. + g_t}, as a float and what it lacks; formed once for every
// (sequence, head, chunk) and kept as [3][64]: c's two floats, dt (0 past the sequence's end).
constexpr int kSdTok = 3 * kSdQ;
template <typename IO>
__device__ __forceinline__ void sd_write_tokens(float *o, const IO *dt, int64_t stride, int64_t t0, int64_t len, float bias,
                                                int softplus, float a2, int lane) {   // one wave, token = lane
    float d = 0.0f;
    if (t0 + lane < len) {
        d = io<IO>::ld(dt, (t0 + lane) * stride) + bias;
        if (softplus) d = softplus_f32(d);
    }
    const double c = wave_incl_sum64((double)(a2 * d));
    const float ch = (float)c;
    o[lane] = ch;
    o[kSdQ + lane] = (float)(c - (double)ch);
    o[2 * kSdQ + lane] = d;
}
// In LDS, with what follows from them (read four tokens at a time, 16 bytes).
struct alignas(16) sd_tokens {
    float ch[kSdQ], cl[kSdQ];
    float dt[kSdQ];
    float w[kSdQ];              // e^{c_last - c_t} dt_t
    float e[kSdQ];              // e^{c_t}
    float dec, pad[3];          // e^{c_last}
};
static_assert(sizeof(sd_tokens) % 16 == 0 && alignof(sd_tokens) == 16, "four tokens in a 16-byte read");
struct sd_tok { float h, l, d; };   // a lane's token
__device__ __forceinline__ sd_tok sd_load_tokens(const float *o, int lane) { return {o[lane], o[kSdQ + lane], o[2 * kSdQ + lane]}; }
__device__ __forceinline__ float sd_stage_tokens(sd_tokens &s, sd_tok v, int lane) {   // one wave; e^{c_last - c_t}
    auto last = [](float x) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), kSdQ - 1)); };
    const float th = last(v.h), tl = last(v.l), r = hw_exp2((th - v.h) + (tl - v.l));
    s.ch[lane] = v.h;
    s.cl[lane] = v.l;
    s.dt[lane] = v.d;
    s.w[lane] = r * v.d;
    s.e[lane] = hw_exp2(v.h + v.l);
    if (lane == 0) s.dec = hw_exp2(th + tl);
    return r;
}
__device__ __forceinline__ f32x4_t ld4(const float *p) { return *reinterpret_cast<const f32x4_t *>(p); }

// ---- the convolution ------------------------------------------------------------------------

// u is rounded in the middle of the path, and every kernel that forms it has to form the same one: the exact value
// rounded to fp32 and then to bf16.  The fp32 value u = silu(v) that conv_silu returns, with v from four products added up
// one after the other and `size` the sum of the sizes of the four sums (v the last), is off by at most
//   1.1 * 2^-24 size               (the sums' roundings; silu's slope is below 1.1)
//   (7 + 2.2 |v|) 2^-24 |u|        (the exponent's roundings, where v < 0; the exponential and the reciprocal, 2 each; a sum,
//                                   a product and v itself, 1 each)
// and `near` says whether a border between two bf16 values is that near (one value in a few thousand): then it is formed
// again in 64 bits.  (Where e^-v leaves fp32, v is near by its size.)
__device__ __forceinline__ float conv_silu(float v, float size, bool &near) {
    const float u = silu_f32(v);
    const float border = __uint_as_float((__float_as_uint(u) & 0xffff0000u) | 0x8000u);
    const float rel = fmaf(fmaxf(-v, 0.0f), 2.5f * 0x1p-24f, 8.0f * 0x1p-24f);
    near = !(fabsf(u - border) > fmaf(size, 1.125f * 0x1p-24f, rel * fabsf(u)));   // (not "<=", so that a NaN is near)
    return u;
}

// (The second rounding on the bits: conversions in a row would be taken as one.)
__device__ __forceinline__ uint16_t silu_bf16_64(double v) {
    const uint32_t b = __float_as_uint((float)(v / (1.0 + exp(-v))));
    if ((b & 0x7fffffffu) > 0x7f800000u) return (uint16_t)(b >> 16 | 0x40u);   // NaN
    return (uint16_t)((b + 0x7fffu + (b >> 16 & 1u)) >> 16);
}

// kSdConvV channels of a row, as raw words; rows of a projected tensor start anywhere (aligned: 4 elements).
template <typename IO, bool AL> struct conv_vec {
    __device__ __forceinline__ static void load(const IO *p, IO (&v)[kSdConvV]) {
        if constexpr (AL) {
            typedef uint32_t words __attribute__((ext_vector_type(sizeof(IO)), may_alias));
            const words w = *reinterpret_cast<const words *>(p);
            __builtin_memcpy(v, &w, sizeof w);
        } else {
#pragma unroll
            for (int k = 0; k < kSdConvV; ++k) v[k] = p[k];
        }
    }
};
// To the layer's own tensors, whose rows hold a multiple of eight elements.
template <typename IO> __device__ __forceinline__ void conv_store(IO *p, const IO (&v)[kSdConvV]) {
    typedef uint32_t words __attribute__((ext_vector_type(sizeof(IO)), may_alias));
    words w;
    __builtin_memcpy(&w, v, sizeof w);
    *reinterpret_cast<words *>(p) = w;
}
template <typename IO> __device__ __forceinline__ float io_f32(IO v) {
    if constexpr (sizeof(IO) == 2) return bf16_to_f32(v);
    else return v;
}

// The taps of kSdConvV channels from c on, oldest first, zeros in front where there are fewer than four.
__device__ __forceinline__ void conv_weights(const float *w, int width, int c, float (&o)[kSdTaps][kSdConvV]) {
    if (width == kSdTaps) {
        typedef float any4 __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
        for (int i = 0; i < kSdConvV; ++i) {
            const any4 v = *reinterpret_cast<const any4 *>(w + (int64_t)(c + i) * kSdTaps);
#pragma unroll
            for (int j = 0; j < kSdTaps; ++j) o[j][i] = v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kSdConvV; ++i)
#pragma unroll
            for (int j = 0; j < kSdTaps; ++j) {
                const int tap = j - (kSdTaps - width);
                o[j][i] = tap >= 0 ? w[(int64_t)(c + i) * width + tap] : 0.0f;
            }
    }
}
__device__ __forceinline__ void conv_bias(const float *b, int c, float (&o)[kSdConvV]) {
    typedef float any4 __attribute__((ext_vector_type(4), aligned(4)));
    any4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (b) v = *reinterpret_cast<const any4 *>(b + c);
#pragma unroll
    for (int i = 0; i < kSdConvV; ++i) o[i] = v[i];
}
// u of a token in its type, from its taps' inputs (oldest first).
template <typename IO>
__device__ __forceinline__ void conv_token(const float (&w)[kSdTaps][kSdConvV], const float (&b)[kSdConvV], const float (&x0)[kSdConvV],
                                           const float (&x1)[kSdConvV], const float (&x2)[kSdConvV], const float (&x3)[kSdConvV],
                                           IO (&o)[kSdConvV]) {
    bool near[kSdConvV] = {};
#pragma unroll
    for (int e = 0; e < kSdConvV; ++e) {
        const float p1 = fmaf(w[0][e], x0[e], b[e]), p2 = fmaf(w[1][e], x1[e], p1), p3 = fmaf(w[2][e], x2[e], p2);
        const float p = fmaf(w[3][e], x3[e], p3);
        if constexpr (sizeof(IO) == 2) {
            o[e] = f32_to_bf16(conv_silu(p, (fabsf(p1) + fabsf(p2)) + (fabsf(p3) + fabsf(p)), near[e]));
        } else {
            o[e] = silu_f32(p);
        }
    }
    if constexpr (sizeof(IO) == 2)
        if (near[0] || near[1] || near[2] || near[3]) {
#pragma unroll 1
            for (int e = 0; e < kSdConvV; ++e)   // (unrolled it takes registers from the rest: B1 L65536 of 4096 channels 263 us for 246, B8 L2048 of 5,248 103 for 96)
                if (near[e]) {
                    double q = fma((double)w[0][e], (double)x0[e], (double)b[e]);
                    q = fma((double)w[1][e], (double)x1[e], q);
                    q = fma((double)w[2][e], (double)x2[e], q);
                    q = fma((double)w[3][e], (double)x3[e], q);
                    o[e] = silu_bf16_64(q);
                }
        }
}

// What a forward's first launch does besides the convolution: the tokens' step sizes and decays.
struct sd_tok_args {
    const void *dt;
    const float *A, *bias;
    float *tok;             // [b][h][chunk][3][64]
    int64_t stride, nchunk;
    int H, softplus, first; // first: the workgroup that starts with them (four heads of a chunk each)
};

// u[b][t][c] = silu(bias + sum_k w[c][k] row_{t - (W-1) + k}), zero at and past a sequence's length; thread:
// kSdConvV channels of `tt` tokens, kSdConvT at a time, the next ones' rows requested before.  A row before token 0 comes
// from st_in (zero without it).  The thread of the first tokens also writes the W - 1 rows before token len
// (st_out may be st_in: nothing else reads it, as tt >= 3).  W4: four taps; fewer count as zeros in front, of rows that count
// as zeros too (what lies in a row that the convolution does not reach, an infinity times no weight, is not its).
// Bound: vector instructions in bf16 (a sixth of the time is the exact rounding's), then HBM: B8 L2048 of 5,248 channels bf16
// 95 us (344 MB, 3.6 TB/s; 80 without the exact rounding), B1 L65536 of 4,096 246 us (1.07 GB, 4.4 TB/s; 203);
// B2 L2048 of 1,664 fp32 16.5 us.  Workgroups behind the convolution's write the tokens' decays, as the work of a launch of
// their own is small.
constexpr int kSdConvT = 4;
template <typename IO, bool AL, bool W4>
__global__ void __launch_bounds__(256)
sd_conv_kernel(const IO *__restrict__ x, int64_t xstride, const float *__restrict__ w, const float *__restrict__ bias,
               int width, const IO *st_in, IO *st_out, const int32_t *__restrict__ lens, IO *__restrict__ u, int64_t L,
               int dc, int tt, int vblocks, int ntiles, sd_tok_args k) {
    if ((int)blockIdx.x >= k.first) {
        const int lane = threadIdx.x & 63, quads = (k.H + 3) / 4;
        const int64_t item = blockIdx.x - k.first;
        const int h = (int)(item % quads) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int64_t c = item / quads % k.nchunk, b = item / quads / k.nchunk;
        if (h >= k.H) return;
        const int64_t len = lens ? min(max((int64_t)lens[b], (int64_t)0), L) : L;
        sd_write_tokens(k.tok + ((b * k.H + h) * k.nchunk + c) * kSdTok, static_cast<const IO *>(k.dt) + b * L * k.stride + h,
                        k.stride, c * kSdQ, len, k.bias ? k.bias[h] : 0.0f, k.softplus, k.A[h] * kLog2e, lane);
        return;
    }
    const int v = blockIdx.x % vblocks * 256 + threadIdx.x;
    if (v >= dc / kSdConvV) return;
    const int c = v * kSdConvV;
    const int64_t b = blockIdx.x / vblocks / ntiles, t0 = (int64_t)(blockIdx.x / vblocks % ntiles) * tt, t1 = min(t0 + tt, L);
    const int64_t len = lens ? min(max((int64_t)lens[b], (int64_t)0), L) : L;
    const IO *xb = x + b * L * xstride + c;
    IO *ub = u + b * L * dc + c;
    const int h = width - 1;
    auto row = [&](int64_t t, IO (&o)[kSdConvV]) {   // t >= -3
        if (t >= 0) conv_vec<IO, AL>::load(xb + t * xstride, o);
        else if (st_in && t >= -h) conv_vec<IO, true>::load(st_in + (b * h + h + t) * dc + c, o);
        else
            for (int i = 0; i < kSdConvV; ++i) o[i] = 0;
    };
    IO r[kSdConvT][kSdConvV] = {};
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < kSdConvT; ++i)
            if (t + i < min(t1, len)) conv_vec<IO, AL>::load(xb + (t + i) * xstride, r[i]);
    };
    fetch(t0);
    float wv[kSdTaps][kSdConvV], bv[kSdConvV], past[kSdTaps - 1][kSdConvV];
    conv_weights(w, width, c, wv);
    conv_bias(bias, c, bv);
#pragma unroll
    for (int j = 0; j < kSdTaps - 1; ++j) {
        IO o[kSdConvV];
        row(t0 - 3 + j, o);
#pragma unroll
        for (int i = 0; i < kSdConvV; ++i) past[j][i] = W4 || h >= 3 - j ? io_f32(o[i]) : 0.0f;
    }
    for (int64_t t = t0; t < t1; t += kSdConvT) {
        IO now[kSdConvT][kSdConvV];
#pragma unroll
        for (int i = 0; i < kSdConvT; ++i)
#pragma unroll
            for (int e = 0; e < kSdConvV; ++e) now[i][e] = r[i][e];
        fetch(t + kSdConvT);
#pragma unroll
        for (int i = 0; i < kSdConvT; ++i) {
            if (t + i >= t1) break;
            IO o[kSdConvV];
            float last[kSdConvV];
#pragma unroll
            for (int e = 0; e < kSdConvV; ++e) last[e] = io_f32(now[i][e]);
            conv_token<IO>(wv, bv, past[0], past[1], past[2], last, o);
#pragma unroll
            for (int e = 0; e < kSdConvV; ++e) {
                past[0][e] = W4 || h >= 3 ? past[1][e] : 0.0f;
                past[1][e] = W4 || h >= 2 ? past[2][e] : 0.0f;
                past[2][e] = W4 || h >= 1 ? last[e] : 0.0f;
            }
            if (t + i >= len)
                for (int e = 0; e < kSdConvV; ++e) o[e] = 0;
            conv_store<IO>(ub + (t + i) * dc, o);
        }
    }
    if (st_out && t0 == 0) {   // (last: st_out may be st_in)
        IO keep[kSdTaps - 1][kSdConvV];
#pragma unroll
        for (int j = 0; j < kSdTaps - 1; ++j)
            if (j < h) row(len - h + j, keep[j]);
#pragma unroll
        for (int j = 0; j < kSdTaps - 1; ++j)
            if (j < h) conv_store<IO>(st_out + (b * h + j) * dc + c, keep[j]);
    }
}

// ---- the layer over a sequence --------------------------------------------------------------

struct sd_shape {
    int64_t L;              // tokens (padded length)
    int H, P, G, N;         // heads, channels per head, groups, states
    int PT;                 // 64-channel tiles per head
    int dc;                 // elements per row of u: H P + 2 G N
    int64_t dt_stride;      // elements between tokens of the step sizes
    int softplus;
    int64_t nchunk;         // chunks of a sequence
    int nseg;               // segments of a sequence, one after the other in workgroups of their own
    int64_t cps;            // chunks per segment
};

// Where workgroup (sequence b, head h, tile pt) finds its rows.
template <typename IO> struct sd_view {
    const IO *x, *B, *C;
    int pw;                 // channels of the tile that exist
    __device__ __forceinline__ sd_view(const IO *u, const sd_shape &s, int64_t b, int h, int pt) {
        const IO *r = u + b * s.L * s.dc;
        const int g = h / (s.H / s.G);
        x = r + h * s.P + pt * 64;
        B = r + s.H * s.P + g * s.N;
        C = B + s.G * s.N;
        pw = min(64, s.P - pt * 64);
    }
};

// State accumulators of a wave: D[n][p], rows n = 16 nb + 4 (lane / 16) + e, column p = 16 w + lane % 16.
// In memory [p][n]: four consecutive n per lane.
template <int NB>
__device__ __forceinline__ void sd_load_state(f32x4_t (&S)[NB], const float *m, int N, int pw, int w, int lane) {
    const int p = 16 * w + (lane & 15);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int n = 16 * nb + 4 * (lane >> 4);
        S[nb] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        if (p < pw && n < N) S[nb] = ld4(m + (int64_t)p * N + n);
    }
}
template <int NB>
__device__ __forceinline__ void sd_store_state(const f32x4_t (&S)[NB], float *m, int N, int pw, int w, int lane) {
    const int p = 16 * w + (lane & 15);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int n = 16 * nb + 4 * (lane >> 4);
        if (p < pw && n < N) *reinterpret_cast<f32x4_t *>(m + (int64_t)p * N + n) = S[nb];
    }
}

// A workgroup's segment: of sequence b, head h, tile pt the chunks [c0, c1), of which [c0, live) have tokens.
struct sd_segment {
    int64_t b, c0, c1, live, len;
    int h, pt, seg;
    __device__ __forceinline__ sd_segment(const sd_shape &s, const int32_t *lens) {
        seg = blockIdx.x % s.nseg;
        pt = blockIdx.x / s.nseg % s.PT;
        h = blockIdx.x / s.nseg / s.PT % s.H;
        b = blockIdx.x / s.nseg / s.PT / s.H;
        len = lens ? min(max((int64_t)lens[b], (int64_t)0), s.L) : s.L;
        c0 = seg * s.cps;
        c1 = min(c0 + s.cps, s.nchunk);
        live = max(c0, min(c1, (len + kSdQ - 1) / kSdQ));
    }
    // element (p, n) = (64 pt, 0) of the tile in [b][h][k of n][P][N]
    __device__ __forceinline__ int64_t state_at(const sd_shape &s, int64_t n, int64_t k) const {
        return (((b * s.H + h) * n + k) * s.P + (int64_t)pt * 64) * s.N;
    }
};

// The states (or adjoints, REV) that the segments start from, from those that they leave when they start from zero:
// one workgroup per 1024 elements of a (sequence, head).  seg: [b][h][segment][P N], in place.  Bound: the chain of
// segments, a read and a write each (B1 L65536 H32 P64 N128, 16 segments: 19 us).
template <bool REV>
__global__ void __launch_bounds__(256)
sd_combine_kernel(const float *__restrict__ tok, const float *__restrict__ first, float *__restrict__ seg, sd_shape s, int blocks) {
    extern __shared__ float dec[];   // nseg decays
    const int64_t bh = blockIdx.x / blocks;
    tok += bh * s.nchunk * kSdTok;
    for (int k = threadIdx.x >> 6; k < s.nseg; k += 4) {   // a wave per segment
        double sum = 0.0;
        for (int64_t c = k * s.cps + (threadIdx.x & 63); c < min((k + 1) * s.cps, s.nchunk); c += 64)
            sum += (double)tok[c * kSdTok + kSdQ - 1] + (double)tok[c * kSdTok + 2 * kSdQ - 1];
#pragma unroll
        for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m, 64);
        if ((threadIdx.x & 63) == 0) dec[k] = hw_exp2((float)sum);
    }
    __syncthreads();
    const int pn = s.P * s.N, e = (blockIdx.x % blocks * 256 + threadIdx.x) * 4;
    if (e >= pn) return;
    f32x4_t cur = first ? ld4(first + bh * pn + e) : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < s.nseg; ++i) {
        const int k = REV ? s.nseg - 1 - i : i;
        float *m = seg + (bh * s.nseg + k) * pn + e;
        const f32x4_t own = ld4(m);
        *reinterpret_cast<f32x4_t *>(m) = cur;
        cur = cur * dec[k] + own;
    }
}

// M in LDS: 64 x 64 without the quarter of t < 32 <= s, which is zero and not read.  32 rows of 32, then 32 of 64 columns.
template <typename E> struct pairs_tile {
    static constexpr int size = 32 * (sd_ld<E>(32) + sd_ld<E>(64));
    __device__ __forceinline__ static int at(int t, bool low) {   // low: t >= 32
        return low ? 32 * sd_ld<E>(32) + (t - 32) * sd_ld<E>(64) : t * sd_ld<E>(32);
    }
    __device__ __forceinline__ static op32<E> row32(const E *m, int j, int k0, int lane) {   // rows of block j
        return j >= 2 ? ssm::row32<E, 64>(m + 32 * sd_ld<E>(32), 16 * j - 32, k0, lane) : ssm::row32<E, 32>(m, 16 * j, k0, lane);
    }
};

// One workgroup per (sequence, head, 64-channel tile, segment): the segment's chunks in order, the state in
// accumulators.  from: the segments' first states [b][h][segment][P][N], or null (zero); last: [b][h][P][N].  ckpt:
// [b][h][chunk][P][N], receives the state entering each chunk, or null.
// FULL: whole tiles (P a multiple of 64, N = NT), without the checks for less (B8 L2048 H80 N64: 192 us, 200 with them; B1
// L65536 H32 N128 402 and 417; no difference where the chunks' states are written).
// The state stays in accumulators, so HBM sees rows and y only (rows through L2 where heads share B and C).  Bound: the
// chain of a chunk's products: the waves wait half of the time (two barriers a chunk), while vector instructions are busy
// 38 % of it and LDS 34 %; B8 L2048 H80 N64 bf16 186 us (rows and y, 340 MB, 1.8 TB/s; reads of C without their bank
// conflicts relieved LDS and changed nothing), with the chunks' states written 253; B1 L65536 H32 N128 in 16
// segments 404; B2 L2048 H24 fp32 45.  Three waves a SIMD (N <= 64, bf16) is what LDS allows.
template <typename E, int NT, bool FULL>
__global__ void __launch_bounds__(kSdThreads)
__attribute__((amdgpu_waves_per_eu(sd<E>::split && NT == 64 ? 3 : 2)))
sd_scan_kernel(const typename sd<E>::io *__restrict__ u_, const float *__restrict__ tok, const float *__restrict__ Dv,
               const int32_t *__restrict__ lens, const float *from, typename sd<E>::io *__restrict__ y_, float *last,
               float *__restrict__ ckpt, sd_shape s) {
    using IO = typename sd<E>::io;
    using F = typename sd<E>::frag;
    constexpr int NB = NT / 16;
    const int N = FULL ? NT : s.N;
    __shared__ __attribute__((aligned(16))) E tB[64 * sd_ld<E>(NT)], tC[64 * sd_ld<E>(NT)], tX[64 * sd_ld<E>(64)];
    __shared__ __attribute__((aligned(16))) E tM[formed<E>::N][pairs_tile<E>::size];
    __shared__ sd_tokens tk;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, q4 = 4 * (lane >> 4);
    const sd_segment at(s, lens);
    const int64_t b = at.b, len = at.len;
    const int h = at.h, pt = at.pt;
    const sd_view<IO> v(u_, s, b, h, pt);
    const int pw = FULL ? 64 : v.pw;
    const E *xs = reinterpret_cast<const E *>(v.x), *Bs = reinterpret_cast<const E *>(v.B), *Cs = reinterpret_cast<const E *>(v.C);
    const float skip = Dv ? Dv[h] : 0.0f;
    tok += (b * s.H + h) * s.nchunk * kSdTok;
    IO *yb = y_ + (b * s.L * s.H + h) * s.P + pt * 64;
    f32x4_t S[NB];
    if (from) {
        sd_load_state(S, from + at.state_at(s, s.nseg, at.seg), N, pw, w, lane);
    } else {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    auto keep = [&](int64_t c) { sd_store_state(S, ckpt + at.state_at(s, s.nchunk, c), N, pw, w, lane); };
    tile64<E, NT> rB, rC;
    tile64<E, 64> rX;
    sd_tok rt = {};
    auto fetch = [&](int64_t t0) {
        const int rows = (int)min((int64_t)64, len - t0);
        rB.load(Bs + t0 * s.dc, s.dc, rows, FULL ? NT : N);
        rC.load(Cs + t0 * s.dc, s.dc, rows, FULL ? NT : N);
        rX.load(xs + t0 * s.dc, s.dc, rows, pw);
        if (w == 0) rt = sd_load_tokens(tok + t0 / kSdQ * kSdTok, lane);
    };
    if (at.c0 < at.live) fetch(at.c0 * kSdQ);
    for (int64_t c = at.c0; c < at.live; ++c) {
        const int64_t t0 = c * kSdQ;
        rB.stage(tB);
        rC.stage(tC);
        rX.stage(tX);
        if (w == 0) sd_stage_tokens(tk, rt, lane);
        if (c + 1 < at.live) fetch(t0 + kSdQ);
        if (ckpt) keep(c);
        __syncthreads();
        // Y^T[p][t] from the state entering, and G^T[s][t] for this wave's 16 tokens s
        f32x4_t Y[4] = {}, Gt[4] = {};
#pragma unroll
        for (int k = 0; k < NB; k += 2) {
            const formed<E> s0(S[k]), s1(S[k + 1]);
            const F b0 = ld_row<E, NT>(tB, 16 * w, 16 * k, lane), b1 = ld_row<E, NT>(tB, 16 * w, 16 * k + 16, lane);
            F c0[4], c1[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c0[j] = ld_row<E, NT>(tC, 16 * j, 16 * k, lane);
                c1[j] = ld_row<E, NT>(tC, 16 * j, 16 * k + 16, lane);
            }
#pragma unroll
            for (int m = 0; m < formed<E>::N; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) Y[j] = mma(s0.p[m], s1.p[m], c0[j], c1[j], Y[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                Gt[j] = mma(b0, b1, c0[j], c1[j], Gt[j]);   // (all four blocks: branches around those before w cost registers and more)
        }
        // M[t][s], D on its diagonal.  Past the diagonal block the decay is taken over the block's last token r, in
        // two factors of at most 1: e^{c_t - c_r} and e^{c_r - c_s} dt_s
        {
            const int s0 = 16 * w + q4;
            const f32x4_t sh = ld4(tk.ch + s0), sl = ld4(tk.cl + s0), sd4 = ld4(tk.dt + s0);
            const float rh = tk.ch[16 * w + 15], rl = tk.cl[16 * w + 15];
            f32x4_t fs;
#pragma unroll
            for (int e = 0; e < 4; ++e) fs[e] = hw_exp2((rh - sh[e]) + (rl - sl[e])) * sd4[e];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 16 * j + c16;
                f32x4_t m = {0.0f, 0.0f, 0.0f, 0.0f};
                if (j > w) {
                    m = Gt[j] * fs * hw_exp2((tk.ch[t] - rh) + (tk.cl[t] - rl));
                } else if (j == w) {
                    const float th = tk.ch[t], tl = tk.cl[t];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float k = hw_exp2((th - sh[e]) + (tl - sl[e]));
                        m[e] = q4 + e <= c16 ? Gt[j][e] * (k * sd4[e]) : 0.0f;
                        if (q4 + e == c16) m[e] += skip;
                    }
                }
                if (j < (w & ~1)) continue;   // (the products read pairs of 16 tokens s up to t's)
                const formed<E> f(m);
#pragma unroll
                for (int i = 0; i < formed<E>::N; ++i) *reinterpret_cast<F *>(&tM[i][pairs_tile<E>::at(t, j >= 2) + s0]) = f.p[i];
            }
        }
        // the state leaving the chunk
        const op32<E> xf[2] = {col32<E, 64>(tX, 0, 16 * w, lane), col32<E, 64>(tX, 32, 16 * w, lane)};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb] *= tk.dec;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float *wt = tk.w + 32 * i + 2 * q4;
            const formed<E> x0(widen(xf[i].lo) * ld4(wt)), x1(widen(xf[i].hi) * ld4(wt + 4));
#pragma unroll
            for (int n0 = 0; n0 < NB; n0 += 4) {
                op32<E> bv[4];
#pragma unroll
                for (int nb = 0; nb < 4; ++nb) bv[nb] = col32<E, NT>(tB, 32 * i, 16 * (n0 + nb), lane);
#pragma unroll
                for (int m = 0; m < formed<E>::N; ++m)
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb) S[n0 + nb] = mma(bv[nb].lo, bv[nb].hi, x0.p[m], x1.p[m], S[n0 + nb]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) Y[j] *= tk.e[16 * j + c16];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int m = 0; m < formed<E>::N; ++m)
#pragma unroll
                for (int j = 2 * i; j < 4; ++j) Y[j] = mma(xf[i], pairs_tile<E>::row32(tM[m], j, 32 * i, lane), Y[j]);
        const int rows = (int)min((int64_t)64, len - t0);
        char *yc = reinterpret_cast<char *>(yb + t0 * s.H * s.P);
        const uint32_t yrow = (uint32_t)(s.H * s.P) * (uint32_t)sizeof(IO), yoff = (uint32_t)c16 * yrow + (uint32_t)(16 * w + q4) * (uint32_t)sizeof(IO);
        auto put = [&](int j, f32x4_t o) {
            char *yp = yc + (yoff + (uint32_t)(16 * j) * yrow);
            if constexpr (sizeof(IO) == 2)
                *reinterpret_cast<u32x2_t *>(yp) = u32x2_t{f32x2_to_bf16x2(o[0], o[1]), f32x2_to_bf16x2(o[2], o[3])};
            else *reinterpret_cast<f32x4_t *>(yp) = o;
        };
        if (rows == 64) {
            if (16 * w + q4 < pw) {
#pragma unroll
                for (int j = 0; j < 4; ++j) put(j, Y[j]);
            }
        } else if (16 * w + q4 < pw) {   // the sequence's last chunk
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (t0 + 16 * j + c16 < s.L) put(j, 16 * j + c16 < rows ? Y[j] : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
        }
    }
    // chunks past the sequence's end: the state stays, y is zero
    for (int64_t c = at.live; c < at.c1; ++c) {
        if (ckpt) keep(c);
        if (16 * w + q4 >= pw) continue;
        for (int j = 0; j < 4; ++j) {
            const int64_t t = c * kSdQ + 16 * j + c16;
            if (t >= s.L) continue;
            IO *yp = yb + t * s.H * s.P + 16 * w + q4;
            for (int e = 0; e < 4; ++e) yp[e] = 0;
        }
    }
    if (last && at.seg == s.nseg - 1) sd_store_state(S, last + at.state_at(s, 1, 0), N, pw, w, lane);
}

// ---- one token ------------------------------------------------------------------------------

// The convolution of one token a sequence, its rows advanced in place; thread: kSdConvV channels of a sequence.
// Bound: its reads' latency (256 sequences of 5,248 channels bf16: 10.6 us, 13.4 MB; one of 4,096: 3.1 us).  The prompt's
// kernel took 24 us: a thread of it reads past tokens and writes the rows after its own work.
template <typename IO, bool AL>
__global__ void __launch_bounds__(256)
sd_conv_step_kernel(const IO *__restrict__ x, int64_t xstride, const float *__restrict__ w, const float *__restrict__ bias,
                    int width, IO *__restrict__ st, IO *__restrict__ u, int dc, int vblocks) {
    const int v = blockIdx.x % vblocks * 256 + threadIdx.x;
    if (v >= dc / kSdConvV) return;
    const int c = v * kSdConvV, h = width - 1;
    const int64_t b = blockIdx.x / vblocks;
    IO r[kSdTaps][kSdConvV] = {}, o[kSdConvV];
    conv_vec<IO, AL>::load(x + b * xstride + c, r[3]);
#pragma unroll
    for (int j = 0; j < kSdTaps - 1; ++j)
        if (j >= kSdTaps - width) conv_vec<IO, true>::load(st + (b * h + j - (kSdTaps - width)) * dc + c, r[j]);
    float wv[kSdTaps][kSdConvV], bv[kSdConvV], xv[kSdTaps][kSdConvV];
    conv_weights(w, width, c, wv);
    conv_bias(bias, c, bv);
#pragma unroll
    for (int j = 0; j < kSdTaps; ++j)
#pragma unroll
        for (int e = 0; e < kSdConvV; ++e) xv[j][e] = io_f32(r[j][e]);
    conv_token<IO>(wv, bv, xv[0], xv[1], xv[2], xv[3], o);
    conv_store<IO>(u + b * dc + c, o);
#pragma unroll
    for (int j = 1; j < kSdTaps; ++j)
        if (j > kSdTaps - width) conv_store<IO>(st + (b * h + j - 1 - (kSdTaps - width)) * dc + c, r[j]);
}

// One workgroup per (sequence, head, part of its channels): LPR lanes hold a channel's N states, four each; U channels
// at a time.  Bound: HBM, the state read and written once (256 sequences of 80 heads P64 N64: 671 MB in 127 us, 5.3 TB/s;
// one of 32 heads N128: 3.9 us, 6.6 with one workgroup a head).
template <typename IO, int LPR, int U>
__global__ void __launch_bounds__(256)
sd_step_kernel(float *__restrict__ state, const IO *__restrict__ u, const IO *__restrict__ dt, int64_t dt_stride,
               const float *__restrict__ A, const float *__restrict__ Dv, const float *__restrict__ dt_bias,
               int softplus, IO *__restrict__ y, int H, int P, int G, int N, int parts) {
    constexpr int ROWS = 256 / LPR;
    const int part = blockIdx.x % (unsigned)parts, h = blockIdx.x / (unsigned)parts % (unsigned)H;
    const int64_t b = blockIdx.x / (unsigned)parts / (unsigned)H;
    const IO *r = u + b * (H * P + 2 * G * N);
    const int g = h / (H / G), n = (threadIdx.x % LPR) * 4;
    float *sb = state + (b * H + h) * P * N;
    const int row = threadIdx.x / LPR;
    const float v = io<IO>::ld(dt, b * dt_stride + h) + (dt_bias ? dt_bias[h] : 0.0f);
    f32x4_t Bv = {0.0f, 0.0f, 0.0f, 0.0f}, Cv = Bv;
    if (n < N) {
        const IO *Bp = r + H * P + g * N + n, *Cp = Bp + G * N;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            Bv[e] = io<IO>::ld(Bp, e);
            Cv[e] = io<IO>::ld(Cp, e);
        }
    }
    const float skip = Dv ? Dv[h] : 0.0f, ah = A[h];
    for (int p0 = part * ROWS * U; p0 < P; p0 += parts * ROWS * U) {
        f32x4_t st[U];
        float x[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int p = p0 + i * ROWS + row;
            if (p < P) {
                x[i] = io<IO>::ld(r, h * P + p);
                if (n < N) st[i] = ld4(sb + (int64_t)p * N + n);
            }
        }
        // a S + in = S + ((a - 1) S + in): a decay near 1 would lose by its rounding what a slow head remembers by
        // (60,000 tokens at a memory of 20,000, the same step size every token: the state off by 1.4e-3 of its rms
        // that way).  Below 1/2 the sum with S would lose more than a does.  (An infinite S stays what it is: the product
        // takes the largest finite value for it.)
        const float d = softplus ? softplus_f32(v) : v, am1 = expm1f(ah * d), a = expf(ah * d);
        const bool slow = __builtin_amdgcn_readfirstlane(am1 > -0.5f);   // (the same in all lanes)
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int p = p0 + i * ROWS + row;
            if (p >= P) continue;   // (a channel's lanes together)
            float o = 0.0f;
            if (n < N) {
                const f32x4_t in = Bv * (d * x[i]);
                if (slow) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        st[i][e] += fmaf(__builtin_amdgcn_fmed3f(st[i][e], -__FLT_MAX__, __FLT_MAX__), am1, in[e]);
                } else {
                    st[i] = st[i] * a + in;
                }
                *reinterpret_cast<f32x4_t *>(sb + (int64_t)p * N + n) = st[i];
                o = st[i][0] * Cv[0] + st[i][1] * Cv[1] + st[i][2] * Cv[2] + st[i][3] * Cv[3];
            }
#pragma unroll
            for (int m = 1; m < LPR; m *= 2) o += __shfl_xor(o, m, 64);
            if (n == 0) io<IO>::st(y, (b * H + h) * P + p, o + skip * x[i]);
        }
    }
}

}  // namespace ssm
