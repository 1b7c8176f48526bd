// The gated linear recurrence, one state per channel:
//
//   log a_t = A[d] sigmoid(r_t)                      (A <= 0: the decay a_t lies in (0, 1])
//   h_t     = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(g_t) x_t
//   y_t     = h_t silu(z_t)                          (z optional)
//
// and its gradients, each in one pass over the data.
//
// Work items.  A sequence is cut into chunks of kGatedChunk tokens and its channels into tiles of
// 64 V (lane = V neighbouring channels); one workgroup takes one (sequence, tile, chunk).  Its
// kGatedWaves waves hold kGatedRows tokens each in registers.  Over a span of tokens the
// recurrence is the map h -> P h + H (P: product of the decays, H: the state reached from zero),
// and maps compose, so that
//   1. every wave forms (P, H) of its tokens,
//   2. wave 0 folds the waves' maps into the chunk's, fetches the state at the chunk's start from
//      the chunks before it (the chain, below) and publishes the state at its end,
//   3. every wave folds the maps of the waves before it onto that state and walks its tokens again
//      from there, writing y.
// The inputs are read once and the outputs written once, whatever the length.
//
// The chain.  word[sequence][chunk][channel] is 64 bits: (P, H) as two floats, P = -1 meaning that
// H is the state itself, all ones meaning that nothing is there yet (the words are filled with ones
// before the kernel starts).  A chunk publishes its map at once and the state at its end as soon as
// it knows it; the two halves travel in one 64-bit store, so a word that is read is whole and
// nothing else has to be ordered.  A chunk reads the kGatedWindow words before its own: with a
// state among them and maps after it, the state at its start is the fold of those maps, oldest
// first, onto that state -- the same operations in the same order whichever word held the state,
// so that the results do not depend on timing.
//
// Every wait ends: an item's number is drawn from a counter when its workgroup starts, and the
// items of a chain are numbered in the order of the chain.  Whoever waits, waits for items that
// started earlier, and the earliest of those waits for nobody.  There is one counter per
// blockIdx mod 8 (the XCDs take workgroups in turn), each with the chains of that residue, so that
// a chain's words stay in one XCD's reach and the counters are not fought over by the whole chip.
#pragma once

#include <float.h>

#include "device_math.h"

namespace ssm {

constexpr int kGatedRows = 8;                            // tokens per wave
constexpr int kGatedWaves = 8;                           // waves per workgroup
constexpr int kGatedChunk = kGatedRows * kGatedWaves;    // tokens per work item
constexpr int kGatedWindow = 4;                          // words of the chain read at a time
constexpr int kGatedGroups = 8;                          // counters (one per XCD)
constexpr int kGatedCounterStride = 64;                  // ints between them: lines of their own

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

// V neighbouring I/O elements of a row as raw 32-bit words.  Rows of an odd width start at odd
// elements, so the accesses assume no more than the element's own alignment (the memory unit takes
// dwords at any byte address).
template <int V, typename IO> struct row_words {
    static constexpr int W = V * (int)sizeof(IO) < 4 ? 1 : V * (int)sizeof(IO) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const IO *p) {
        if constexpr (V * sizeof(IO) < 4) {
            w[0] = *p;
        } else {
            typedef uint32_t any_u32 __attribute__((ext_vector_type(W), aligned(sizeof(IO))));
            const any_u32 v = __builtin_nontemporal_load(reinterpret_cast<const any_u32 *>(p));
            __builtin_memcpy(w, &v, sizeof w);
        }
    }
    __device__ __forceinline__ float get(int v) const {
        if constexpr (sizeof(IO) == 4) return __uint_as_float(w[v]);
        else return __uint_as_float((v & 1) ? (w[v >> 1] & 0xffff0000u) : (w[v >> 1] << 16));
    }
    __device__ __forceinline__ static void store(IO *p, const float (&y)[V]) {
        if constexpr (V * sizeof(IO) < 4) {
            io<IO>::st(p, 0, y[0]);
        } else {
            uint32_t o[W];
            if constexpr (sizeof(IO) == 2) {
#pragma unroll
                for (int i = 0; i < W; ++i) o[i] = f32x2_to_bf16x2(y[2 * i], y[2 * i + 1]);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) o[i] = __float_as_uint(y[i]);
            }
            typedef uint32_t any_u32 __attribute__((ext_vector_type(W), aligned(sizeof(IO))));
            any_u32 v;
            __builtin_memcpy(&v, o, sizeof o);
            __builtin_nontemporal_store(v, reinterpret_cast<any_u32 *>(p));
        }
    }
};

// The chain's words.
constexpr uint32_t kWordEmpty = 0xffffffffu;
__device__ __forceinline__ uint64_t chain_word(float P, float H) {
    const uint32_t p = P != P ? 0x7fc00000u : __float_as_uint(P);   // (a NaN's bits could read as "empty")
    return ((uint64_t)p << 32) | __float_as_uint(H);
}
__device__ __forceinline__ void chain_put(uint64_t *w, float P, float H) {
    __hip_atomic_store(w, chain_word(P, H), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The state that the items before this one leave, for the lane's V channels: the words of items
// first, first + step, ... are read, kGatedWindow of them, stopping at item `end` (which needs
// nobody and publishes a state); stride: words between two items.  One wave.
template <int V>
__device__ __forceinline__ void chain_get(const uint64_t *base, int64_t stride, int first, int step, int end, bool act,
                                          float (&carry)[V]) {
    for (;;) {
        uint64_t w[kGatedWindow][V];
#pragma unroll
        for (int k = 0; k < kGatedWindow; ++k) {
            const int j = step < 0 ? max(first - k, end) : min(first + k, end);
#pragma unroll
            for (int v = 0; v < V; ++v)
                w[k][v] = __hip_atomic_load(const_cast<uint64_t *>(base + j * stride + v), __ATOMIC_RELAXED,
                                            __HIP_MEMORY_SCOPE_AGENT);
        }
        bool all = true;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            bool ok = false;
            float h = 0.0f;
#pragma unroll
            for (int k = kGatedWindow - 1; k >= 0; --k) {   // oldest first
                const uint32_t p = (uint32_t)(w[k][v] >> 32);
                const float H = __uint_as_float((uint32_t)w[k][v]);
                const bool state = p == __float_as_uint(-1.0f);
                h = state ? H : fmaf(__uint_as_float(p), h, H);
                ok = state || (ok && p != kWordEmpty);
            }
            carry[v] = h;
            all = all && ok;
        }
        if (__all(all || !act)) return;
        __builtin_amdgcn_s_sleep(1);
    }
}

// Which item this workgroup takes: (chain, position along the chain), or chain < 0 for none.
// Chains of one residue are walked together, position by position.
struct GatedItem {
    int chain, pos;
};
__device__ __forceinline__ GatedItem gated_item(int chains, int nchunk, int *counters, int *slot) {
    const int q = (int)blockIdx.x % kGatedGroups;
    const int nq = (chains - q + kGatedGroups - 1) / kGatedGroups;
    int n = (int)blockIdx.x / kGatedGroups;
    if (counters) {   // (one chunk per sequence: no chain, any order will do)
        if (threadIdx.x == 0)
            *slot = __hip_atomic_fetch_add(&counters[q * kGatedCounterStride], 1, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        n = __builtin_amdgcn_readfirstlane(*slot);
    }
    if (nq <= 0 || n >= nq * nchunk) return {-1, 0};
    const int pos = n / nq;
    return {(n - pos * nq) * kGatedGroups + q, pos};
}

// Fills the chain's words with ones and clears the counters behind them.
static __global__ void __launch_bounds__(256)
gated_clear_kernel(uint64_t *__restrict__ words, int64_t n, int *__restrict__ counters) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) words[i] = ~uint64_t(0);
    else if (i - n < kGatedGroups * kGatedCounterStride) counters[i - n] = 0;
}

// A token's coefficients for one channel.
struct GatedCoeff {
    float s, i, y, a, q;   // sigmoid(r), sigmoid(g), log2 a, a, 1 - a^2
};
__device__ __forceinline__ GatedCoeff gated_coeff(float r, float g, float a2) {
    GatedCoeff c;
    c.s = sigmoid_f32(r);
    c.i = sigmoid_f32(g);
    c.y = a2 * c.s;
    c.a = hw_exp2(c.y);
    c.q = one_minus_square(c.y, c.a);
    return c;
}

// OUT: y and last_state are written; otherwise only the chain's words (the states at the chunks'
// ends, for the backward pass).
template <typename IO, int V, bool OUT>
__global__ void __launch_bounds__(64 * kGatedWaves)
gated_scan_kernel(const IO *__restrict__ x, const IO *__restrict__ r, const IO *__restrict__ g,
                  const float *__restrict__ A, const IO *__restrict__ z, const float *h0,
                  const int32_t *__restrict__ seq_lens, IO *__restrict__ y, float *last, uint64_t *words,
                  int *counters, int64_t L, int64_t D, int tiles, int chains, int nchunk) {
    constexpr int T = kGatedRows, K = kGatedWaves, C = kGatedChunk;
    using Row = row_words<V, IO>;
    __shared__ float s_P[K][64 * V], s_H[K][64 * V], s_in[64 * V];
    __shared__ int s_slot;
    const GatedItem it = gated_item(chains, nchunk, counters, &s_slot);
    if (it.chain < 0) return;
    const int b = it.chain / tiles, c = it.pos;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The lane's first channel.  Of an odd width the last lane takes the last V channels: those it
    // shares with its neighbour get the same values from both.
    const int64_t dl = (int64_t)(it.chain - b * tiles) * 64 * V + lane * V;
    const bool act = dl < D;
    const int64_t d = min(dl, D - V);
    const int64_t Lb = seq_lens ? min((int64_t)max(seq_lens[b], 0), L) : L;
    const int64_t t0 = (int64_t)c * C + w * T;
    const int64_t row0 = (int64_t)b * L;
    const int nlive = (int)((Lb + C - 1) / C);   // chunks of this sequence that hold tokens

    if (c >= nlive) {   // past the sequence's end
        if constexpr (OUT) {
            if (act) {
                const float zero[V] = {};
                for (int64_t t = t0; t < min(t0 + T, L); ++t) Row::store(y + (row0 + t) * D + d, zero);
                if (last && c == 0 && w == 0)
                    for (int v = 0; v < V; ++v) last[(int64_t)b * D + d + v] = h0 ? h0[(int64_t)b * D + d + v] : 0.0f;
            }
        }
        return;
    }

    // every load of the wave first (rows past the end: the last row again)
    Row rr[T], rg[T], rx[T], rz[OUT ? T : 1];
#pragma unroll
    for (int k = 0; k < T; ++k) {
        const int64_t e = (row0 + min(t0 + k, Lb - 1)) * D + d;
        rr[k].load(r + e);
        rg[k].load(g + e);
        rx[k].load(x + e);
    }
    if constexpr (OUT) {
        if (z) {
#pragma unroll
            for (int k = 0; k < T; ++k) rz[k].load(z + (row0 + min(t0 + k, Lb - 1)) * D + d);
        }
    }
    float a2[V];
#pragma unroll
    for (int v = 0; v < V; ++v) a2[v] = A[d + v] * kLog2e;

    // 1. the coefficients (a token past the end is the identity) and the wave's map
    float a[T][V], bb[T][V], P[V], H[V];
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.0f, H[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < T; ++k) {
        const bool live = t0 + k < Lb;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const GatedCoeff cf = gated_coeff(rr[k].get(v), rg[k].get(v), a2[v]);
            a[k][v] = live ? cf.a : 1.0f;
            bb[k][v] = live ? __builtin_amdgcn_sqrtf(cf.q) * cf.i * rx[k].get(v) : 0.0f;
            P[v] *= a[k][v];
            H[v] = fmaf(a[k][v], H[v], bb[k][v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s_P[w][lane * V + v] = P[v];
        s_H[w][lane * V + v] = H[v];
    }
    __syncthreads();

    // 2. the chunk's map, the state at its start, the state at its end
    if (w == 0) {
        float in[V];
        uint64_t *word = words + ((int64_t)b * nchunk + c) * D + d;
        const bool ends = c == nlive - 1;
#pragma unroll
        for (int k = 1; k < K; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float p = s_P[k][lane * V + v];
                H[v] = fmaf(p, H[v], s_H[k][lane * V + v]);
                P[v] *= p;
            }
        if (c == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) in[v] = h0 ? h0[(int64_t)b * D + d + v] : 0.0f;
        } else {
            if (act && !ends) {
#pragma unroll
                for (int v = 0; v < V; ++v) chain_put(word + v, P[v], H[v]);
            }
            chain_get<V>(words + (int64_t)b * nchunk * D + d, D, c - 1, -1, 0, act, in);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float out = fmaf(P[v], in[v], H[v]);
            s_in[lane * V + v] = in[v];
            if (act) {
                if (!ends) chain_put(word + v, -1.0f, out);
                else if (OUT && last) last[(int64_t)b * D + d + v] = out;
            }
        }
    }
    if constexpr (OUT) {
        __syncthreads();
        // 3. the state at the wave's start, and its tokens from there
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = s_in[lane * V + v];
        for (int k = 0; k < w; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(s_P[k][lane * V + v], h[v], s_H[k][lane * V + v]);
#pragma unroll
        for (int k = 0; k < T; ++k) {
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[v] = fmaf(a[k][v], h[v], bb[k][v]);
                o[v] = z ? h[v] * silu_f32(rz[k].get(v)) : h[v];
                if (t0 + k >= Lb) o[v] = 0.0f;
            }
            if (act && t0 + k < L) Row::store(y + (row0 + t0 + k) * D + d, o);
        }
    }
}

// The gradients.  lambda_t = dh_t + G_t with G_t = a_{t+1} lambda_{t+1}, dh_t = dy_t silu(z_t), is
// the same kind of recurrence run from the end (the map of a span is G -> P G + H' with the same
// P), so the items and the chain are the forward's in the other order; the states come from the
// words that the forward left (the state at the end of every chunk).  Each wave forms both maps of
// its tokens, then walks them forwards for the states and backwards for the gradients.  The
// coefficients that cost transcendentals (both sigmoids, the decay) stay in registers in between;
// 1 - a^2 is formed again.  dA's share of the item goes to part[item], summed afterwards in order.
template <typename IO, int V>
__global__ void __launch_bounds__(64 * kGatedWaves)
gated_bwd_kernel(const IO *__restrict__ x, const IO *__restrict__ r, const IO *__restrict__ g,
                 const float *__restrict__ A, const IO *__restrict__ z, const float *__restrict__ h0,
                 const int32_t *__restrict__ seq_lens, const IO *__restrict__ dy, const float *__restrict__ dlast,
                 const uint64_t *__restrict__ states, IO *__restrict__ dx, IO *__restrict__ dr, IO *__restrict__ dg,
                 IO *__restrict__ dz, float *__restrict__ part, float *__restrict__ dh0, uint64_t *words,
                 int *counters, int64_t L, int64_t D, int tiles, int chains, int nchunk) {
    constexpr int T = kGatedRows, K = kGatedWaves, C = kGatedChunk;
    using Row = row_words<V, IO>;
    __shared__ float s_P[K][64 * V], s_H[K][64 * V], s_G[K][64 * V], s_in[64 * V];
    __shared__ int s_slot;
    const GatedItem it = gated_item(chains, nchunk, counters, &s_slot);
    if (it.chain < 0) return;
    const int b = it.chain / tiles, c = nchunk - 1 - it.pos;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t dl = (int64_t)(it.chain - b * tiles) * 64 * V + lane * V;
    const bool act = dl < D;
    const int64_t d = min(dl, D - V);
    const int64_t Lb = seq_lens ? min((int64_t)max(seq_lens[b], 0), L) : L;
    const int64_t t0 = (int64_t)c * C + w * T;
    const int64_t row0 = (int64_t)b * L;
    const int64_t ch = (int64_t)b * D + d;                      // the channel's place in [batch][dim]
    const int64_t item = ((int64_t)b * nchunk + c) * D + d;     // and in [batch][chunk][dim]
    const int nlive = (int)((Lb + C - 1) / C);

    if (c >= nlive) {
        if (act) {
            const float zero[V] = {};
            for (int64_t t = t0; t < min(t0 + T, L); ++t) {
                const int64_t e = (row0 + t) * D + d;
                Row::store(dx + e, zero);
                Row::store(dr + e, zero);
                Row::store(dg + e, zero);
                if (z) Row::store(dz + e, zero);
            }
            if (w == 0)
                for (int v = 0; v < V; ++v) {
                    part[item + v] = 0.0f;
                    if (c == 0 && dh0) dh0[ch + v] = dlast ? dlast[ch + v] : 0.0f;
                }
        }
        return;
    }

    Row rr[T], rg[T], rx[T], ry[T], rz[T];
#pragma unroll
    for (int k = 0; k < T; ++k) {
        const int64_t e = (row0 + min(t0 + k, Lb - 1)) * D + d;
        rr[k].load(r + e);
        rg[k].load(g + e);
        rx[k].load(x + e);
        ry[k].load(dy + e);
    }
    if (z) {
#pragma unroll
        for (int k = 0; k < T; ++k) rz[k].load(z + (row0 + min(t0 + k, Lb - 1)) * D + d);
    }
    float Ad[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Ad[v] = A[d + v];
        // the state at the chunk's start (the low half of the word of the chunk before it)
        h[v] = c == 0 ? (h0 ? h0[ch + v] : 0.0f) : __uint_as_float((uint32_t)states[item - D + v]);
    }

    // 1. the coefficients and the wave's two maps
    float s[T][V], i[T][V], a[T][V], bb[T][V], P[V], H[V], G[V];
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.0f, H[v] = 0.0f, G[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < T; ++k) {
        const bool live = t0 + k < Lb;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const GatedCoeff cf = gated_coeff(rr[k].get(v), rg[k].get(v), Ad[v] * kLog2e);
            s[k][v] = cf.s;
            i[k][v] = cf.i;
            a[k][v] = live ? cf.a : 1.0f;
            bb[k][v] = live ? __builtin_amdgcn_sqrtf(cf.q) * cf.i * rx[k].get(v) : 0.0f;
            P[v] *= a[k][v];
            H[v] = fmaf(a[k][v], H[v], bb[k][v]);
        }
    }
    auto grad_in = [&](int k, int v) {   // dh_t
        const float dyv = ry[k].get(v);
        return t0 + k < Lb ? (z ? dyv * silu_f32(rz[k].get(v)) : dyv) : 0.0f;
    };
#pragma unroll
    for (int k = T - 1; k >= 0; --k)
#pragma unroll
        for (int v = 0; v < V; ++v) G[v] = a[k][v] * (grad_in(k, v) + G[v]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s_P[w][lane * V + v] = P[v];
        s_H[w][lane * V + v] = H[v];
        s_G[w][lane * V + v] = G[v];
    }
    __syncthreads();

    // 2. the adjoint at the chunk's end, and the one that it hands on
    if (w == 0) {
        float in[V], PC[V], GC[V];
        const bool starts = c == nlive - 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            PC[v] = s_P[K - 1][lane * V + v];
            GC[v] = s_G[K - 1][lane * V + v];
        }
#pragma unroll
        for (int k = K - 2; k >= 0; --k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float p = s_P[k][lane * V + v];
                GC[v] = fmaf(p, GC[v], s_G[k][lane * V + v]);
                PC[v] *= p;
            }
        if (starts) {
#pragma unroll
            for (int v = 0; v < V; ++v) in[v] = dlast ? dlast[ch + v] : 0.0f;
        } else {
            if (act && c > 0) {
#pragma unroll
                for (int v = 0; v < V; ++v) chain_put(words + item + v, PC[v], GC[v]);
            }
            chain_get<V>(words + (int64_t)b * nchunk * D + d, D, c + 1, 1, nlive - 1, act, in);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float out = fmaf(PC[v], in[v], GC[v]);
            s_in[lane * V + v] = in[v];
            if (act) {
                if (c > 0) chain_put(words + item + v, -1.0f, out);
                else if (dh0) dh0[ch + v] = out;
            }
        }
    }
    __syncthreads();

    // 3. the states before the wave's tokens (over bb), the adjoint after its last, the gradients
    for (int k = 0; k < w; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(s_P[k][lane * V + v], h[v], s_H[k][lane * V + v]);
    float hT[V];
#pragma unroll
    for (int v = 0; v < V; ++v) G[v] = s_in[lane * V + v];
    for (int k = K - 1; k > w; --k)
#pragma unroll
        for (int v = 0; v < V; ++v) G[v] = fmaf(s_P[k][lane * V + v], G[v], s_G[k][lane * V + v]);
#pragma unroll
    for (int k = 0; k < T; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float hn = fmaf(a[k][v], h[v], bb[k][v]);
            bb[k][v] = h[v];
            h[v] = hn;
        }
#pragma unroll
    for (int v = 0; v < V; ++v) hT[v] = h[v];
    float dA[V] = {};
#pragma unroll
    for (int k = T - 1; k >= 0; --k) {
        float ox[V], og[V], orr[V], oz[V];
        const bool live = t0 + k < Lb;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float xv = rx[k].get(v), dyv = ry[k].get(v);
            float dh = dyv;
            if (z) {   // silu(z) = z sz, silu'(z) = sz (1 + z (1 - sz))
                const float zz = rz[k].get(v), sz = sigmoid_f32(zz);
                oz[v] = live ? dyv * hT[v] * (sz * fmaf(zz, 1.0f - sz, 1.0f)) : 0.0f;
                dh *= zz * sz;
            }
            const float lam = live ? dh + G[v] : G[v];
            G[v] = a[k][v] * lam;
            const float q = one_minus_square(Ad[v] * kLog2e * s[k][v], a[k][v]);
            // 1 / beta; where 1 - a^2 is zero (or below what the unit resolves) the terms with it are dropped
            const float rb = fabsf(q) < FLT_MIN ? 0.0f : __builtin_amdgcn_rsqf(q);
            const float ix = i[k][v] * xv;
            const float lb = lam * (q * rb);             // lambda beta
            const float dla = fmaf(G[v], bb[k][v], -(lam * ix) * (a[k][v] * a[k][v] * rb));
            const float ds = live ? dla * s[k][v] : 0.0f;
            dA[v] += ds;
            orr[v] = ds * (Ad[v] * (1.0f - s[k][v]));
            ox[v] = live ? lb * i[k][v] : 0.0f;
            og[v] = live ? lb * ix * (1.0f - i[k][v]) : 0.0f;
            hT[v] = bb[k][v];
        }
        if (act && t0 + k < L) {
            const int64_t e = (row0 + t0 + k) * D + d;
            Row::store(dx + e, ox);
            Row::store(dr + e, orr);
            Row::store(dg + e, og);
            if (z) Row::store(dz + e, oz);
        }
    }
    __syncthreads();   // (the maps are read)
#pragma unroll
    for (int v = 0; v < V; ++v) s_P[w][lane * V + v] = dA[v];
    __syncthreads();
    if (w == 0 && act) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float t = s_P[0][lane * V + v];
#pragma unroll
            for (int k = 1; k < K; ++k) t += s_P[k][lane * V + v];
            part[item + v] = t;
        }
    }
}

// out[d] = sum of the n rows of part, in an order of their own: 16 waves take every 16th row, and
// their sums are added in order.
constexpr int kColumnWaves = 16;
static __global__ void __launch_bounds__(64 * kColumnWaves)
column_sum_kernel(const float *__restrict__ part, float *__restrict__ out, int64_t n, int64_t D) {
    __shared__ float red[kColumnWaves][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t d = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (d < D)
        for (int64_t k = w; k < n; k += kColumnWaves) s += part[k * D + d];
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && d < D) {
#pragma unroll
        for (int k = 1; k < kColumnWaves; ++k) s += red[k][lane];
        out[d] = s;
    }
}

// One token of every sequence, the state updated in place.
template <typename IO>
__global__ void __launch_bounds__(256)
gated_step_kernel(float *__restrict__ state, const IO *__restrict__ x, const IO *__restrict__ r,
                  const IO *__restrict__ g, const float *__restrict__ A, const IO *__restrict__ z,
                  IO *__restrict__ y, int64_t n, int64_t D) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= n) return;
    const GatedCoeff cf = gated_coeff(io<IO>::ld(r, e), io<IO>::ld(g, e), A[e % D] * kLog2e);
    const float h = fmaf(cf.a, state[e], __builtin_amdgcn_sqrtf(cf.q) * cf.i * io<IO>::ld(x, e));
    state[e] = h;
    io<IO>::st(y, e, z ? h * silu_f32(io<IO>::ld(z, e)) : h);
}

}  // namespace ssm
