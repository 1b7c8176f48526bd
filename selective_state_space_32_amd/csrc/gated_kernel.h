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
// and maps compose.  P is carried as its logarithm, the sum of log2 a: products of decays near 1 are rounded
// with a mean (1 - a of both is a few thousand ulps of 1, and their product is cut off), which slow channels
// add up (the last state of 30,000 tokens at 1 / (1 - a) = 20,000 was off by 1.1e-4 of the rms).  So
//   1. every wave forms (P, H) of its tokens,
//   2. wave 0 folds the waves' maps into the chunk's, fetches the state at the chunk's start from
//      the chunks before it (the chain, below) and publishes the state at its end,
//   3. every wave folds the maps of the waves before it onto that state and walks its tokens again
//      from there, writing y.
// The inputs are read once and the outputs written once, whatever the length.
//
// Bound: HBM.  Per element the forward moves 8 bytes in bf16 (10 with a gate) and issues 43 VALU
// instructions with its gate, 8 of them transcendental (three sigmoids, the decay, a root), which keeps
// the VALU busy for two thirds of its time; the backward moves 14 (18), issues 84 and keeps it as busy.
// Measured (averages at settled clocks), where a copy of 1 GiB reaches 5.1 TB/s: B8 L2048 D5120 bf16 gated
// 167 us for 839 MB (855 by the counters), its backward 305 us for 1,510 MB (1,537); B1 L131072 D2048 bf16
// 410 us for 2,148 MB; B2 L2048 D1536 fp32 25 us for 101 MB, its backward 39 us for 176 MB.  Short
// launches are bound by their latency: 4.5 us for one chunk in four tiles, its backward 6.8.
//
// The split.  Eight tokens per wave keep a lane's values of V channels in registers (72 registers in
// the forward, three workgroups per CU; 128 in the backward, two), and several workgroups per CU let
// one load while another computes or waits.  At B8 L2048 D5120, sixteen waves of eight tokens took
// 221 us where eight of eight took 169 (an earlier form of this kernel); eight of sixteen are an item of two
// chunks, taken for long chains.
//
// The chain.  The state goes from chunk to chunk through memory.  With many chains every chunk waits for
// the one before it (chain_hand): state[sequence][chunk][channel], four bytes, all ones meaning that
// nothing is there yet; the forward's are also the states that the backward starts from.  With few
// chains a round trip per chunk would be all that happens, so the chunks of a chain form groups (the
// host chooses their size; chain_step): word[sequence][item][channel] is 64 bits, a chunk publishes
// its map (log2 P, H), two floats, as soon as it has it, and the last chunk of a group publishes instead the
// state at its end, as (1, h), once it knows it.  A chunk fetches the maps of the chunks before it in
// its group (which wait for nobody; the waves share them), composes them, and applies them to the
// state that the group before left.  Only the groups' last chunks wait in line.  The chain's first
// chunk publishes the constant map (-infinity, state at its end): it alone reads the initial state.
// The words are filled with ones before the kernel starts.  A word travels in one store, so one that is
// read is whole and nothing else has to be ordered.  Which words a chunk combines, and in which order,
// is fixed: the results do not depend on timing.
//
// Every wait ends: an item's number is drawn from a counter when its workgroup starts, and the items
// of a chain are numbered in the order of the chain.  Whoever waits, waits for items that started
// earlier, and the earliest of those waits for nobody.  There are up to kGatedQueues counters (one
// alone is fought over by the whole chip: 768 workgroups that start together wait 9 us), each with an
// equal run of the chains; `run` consecutive workgroups draw from the same one.  The XCDs take
// workgroups in turn, so with eight queues and run = 1 a queue's chains stay in one XCD: its hand-overs
// are the fastest, and neighbouring tiles, which share lines where rows do not start on one, meet in
// its L2 (B8 L2048 D5119 bf16 backward: 368 us, 429 with run = 8).  With run = 8 every XCD works on all
// the chains, where with run = 1 it reads the same few columns of every row, which lie in few of the
// memory's channels (B1 L131072 D2048 bf16 gated: 534 against 475 us).
#pragma once

#include <float.h>

#include "device_math.h"

namespace ssm {

constexpr int kGatedRows = 8;                            // tokens per wave
constexpr int kGatedWaves = 8;                           // waves per workgroup
constexpr int kGatedChunk = kGatedRows * kGatedWaves;    // tokens per stored state (and per item of the backward)
constexpr int kGatedGroup = 64;                          // most items of a chain that share a hand-over
constexpr int kGatedQueues = 8;                          // counters, at most (one per XCD)
constexpr int kGatedRun = 8;                             // workgroups in a row at a counter, or one
constexpr int kGatedCounterStride = 64;                  // ints between them: lines of their own

// u = 1 - a = -expm1(ln 2 y), given y = log2(a) <= 0 and 2^y.  Near a = 1 the difference loses every digit
// that 2^y was rounded in, so there a polynomial in y takes its place, y (c0 + c1 y + ...), interpolated at
// Chebyshev nodes of the interval: degree 4 for a > 0.82 where both the inputs and the outputs are fp32
// (relative error below 1e-9, 1.1e-7 as it is evaluated; the difference below that 3e-7), or degree 2 for
// a > 0.94 (4e-7; the difference 9e-7).  From u come
//   1 - a^2 = u + u a,
//   a       = 1 - u, rounded once, where it matters (gated_coeff): 2^y of the exponential unit is good to an
//             ulp, but near 1 its error has a mean (-7e-9 for 1 - a below 2e-3), which a slow channel adds up
//             over its memory of 1 / (1 - a) tokens wherever decays are all that a state goes on by, whereas an
//             error relative to u is only that error of the state.
template <typename IO> constexpr float kNearOne = sizeof(IO) == 4 ? -0.289f : -0.09f;   // y from which u is near
template <typename IO> __device__ __forceinline__ float one_minus(float y, float exp2_y) {
    float p;
    if constexpr (sizeof(IO) == 4) {
        p = fmaf(y, -1.2270708102732897e-3f, -9.591649286448956e-3f);
        p = fmaf(p, y, -5.550139397382736e-2f);
        p = fmaf(p, y, -0.2402264028787613f);
        p = fmaf(p, y, -0.6931471824645996f);
    } else {
        p = fmaf(y, -5.4223693907260895e-2f, -0.24018345773220062f);
        p = fmaf(p, y, -0.6931469440460205f);
    }
    return y > kNearOne<IO> ? p * y : 1.0f - exp2_y;
}
// 2^y, the decay over a span of tokens.
__device__ __forceinline__ float decay(float y) {
    const float e = hw_exp2(y), u = one_minus<float>(y, e);
    return y > kNearOne<float> ? 1.0f - u : e;
}

// V neighbouring I/O elements of a row as raw 32-bit words.  Rows of an odd width start at odd
// elements, so the accesses assume no more than the element's own alignment (the memory unit takes
// dwords at any byte address).  NT: past the caches, as data that is used once; not where rows start
// inside a line, whose other part a neighbouring tile wants (B8 L2048 D5119 bf16: 199 us through the
// caches, 205 past them, backward 368 and 484; at D5120 185 and 166, 310 and 304).
#define SSM_GLOBAL __attribute__((address_space(1)))   // memory of the device: no other kind is tried
template <int V, typename IO, bool NT = true> struct row_words {
    static constexpr int W = V * (int)sizeof(IO) < 4 ? 1 : V * (int)sizeof(IO) / 4;
    uint32_t w[W];
    // base: the same for the wave; ofs: the lane's byte offset from it -- the memory instructions take the
    // two as they are.
    __device__ __forceinline__ void load(const IO *base, uint32_t ofs) {
        const SSM_GLOBAL char *p = (const SSM_GLOBAL char *)base + ofs;
        if constexpr (V * sizeof(IO) < 4) {
            w[0] = *(const SSM_GLOBAL IO *)p;
        } else {
            typedef uint32_t any_u32 __attribute__((ext_vector_type(W), aligned(sizeof(IO))));
            any_u32 v;
            if constexpr (NT) v = __builtin_nontemporal_load((const SSM_GLOBAL any_u32 *)p);
            else v = *(const SSM_GLOBAL any_u32 *)p;
            __builtin_memcpy(w, &v, sizeof w);
        }
    }
    __device__ __forceinline__ float get(int v) const {
        if constexpr (sizeof(IO) == 4) return __uint_as_float(w[v]);
        else return __uint_as_float((v & 1) ? (w[v >> 1] & 0xffff0000u) : (w[v >> 1] << 16));
    }
    __device__ __forceinline__ void fill(uint32_t v) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = v;
    }
    // The words as if written anew: nothing computed from them before is known to hold after.
    __device__ __forceinline__ void opaque() {
#pragma unroll
        for (int i = 0; i < W; ++i) asm volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ static void store(IO *base, uint32_t ofs, const float (&y)[V]) {
        asm("" : "+v"(ofs));   // (or the offset is widened, and added, ahead of the branch that this is in)
        SSM_GLOBAL char *p = (SSM_GLOBAL char *)base + ofs;
        if constexpr (V * sizeof(IO) < 4) {
            *(SSM_GLOBAL IO *)p = (IO)f32x2_to_bf16x2(y[0], 0.0f);
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
            if constexpr (NT) __builtin_nontemporal_store(v, (SSM_GLOBAL any_u32 *)p);
            else *(SSM_GLOBAL any_u32 *)p = v;
        }
    }
};

// The words of -infinity.
template <typename IO> __device__ __forceinline__ uint32_t minus_inf_words() {
    return sizeof(IO) == 4 ? 0xff800000u : 0xff80ff80u;
}

// The chain's words.
constexpr uint32_t kWordEmpty = 0xffffffffu;
__device__ __forceinline__ uint64_t chain_word(float Y, float H) {
    const uint32_t y = Y != Y ? 0x7fc00000u : __float_as_uint(Y);   // (a NaN's bits could read as "empty")
    return ((uint64_t)y << 32) | __float_as_uint(H);
}
__device__ __forceinline__ void chain_put(uint64_t *w, float Y, float H) {
    __hip_atomic_store(w, chain_word(Y, H), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t chain_read(const uint64_t *w) {
    return __hip_atomic_load(const_cast<uint64_t *>(w), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The chain's step for the item at position pos, called by the whole workgroup: base + p * stride is
// the word of position p (the lane's first of V channels), h -> 2^Y h + H the item's map and start the state
// at position 0's start (both read in wave 0 only; 0 at other positions), `ends`: nobody comes after.
// Leaves the state at the item's start in s_in (behind a barrier) and the one at its end in wave 0's `out`.
template <int V>
__device__ __forceinline__ void chain_step(uint64_t *base, int64_t stride, int pos, int group, bool ends, bool act,
                                           int lane, int w, const float (&Y)[V], const float (&H)[V],
                                           const float (&start)[V], float (&s_map)[3][kGatedWaves][64 * V],
                                           float (&s_in)[64 * V], float (&out)[V]) {
    const int g = pos & (group - 1);   // (a power of two)
    uint64_t *own = base + pos * stride;
    if (w == 0 && act && !ends && g != group - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (pos == 0) chain_put(own + v, -__builtin_inff(), fmaf(decay(Y[v]), start[v], H[v]));
            else chain_put(own + v, Y[v], H[v]);
    }
    // the maps of the group's items before this one, in equal runs over the waves: each composes its run
    const int m = (g + kGatedWaves - 1) / kGatedWaves, lo = w * m, hi = min(lo + m, g);
    if (lo < hi) {
        const uint64_t *src = base + (pos - g + lo) * stride;
        float cy[V], ch[V];
        for (int k = lo; k < hi; ++k, src += stride) {
            uint64_t u[V];
            for (;;) {
                bool all = true;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    u[v] = chain_read(src + v);
                    all = all && (uint32_t)(u[v] >> 32) != kWordEmpty;
                }
                if (__all(all || !act)) break;
                __builtin_amdgcn_s_sleep(1);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float y = __uint_as_float((uint32_t)(u[v] >> 32)), h = __uint_as_float((uint32_t)u[v]);
                ch[v] = k == lo ? h : fmaf(decay(y), ch[v], h);
                cy[v] = k == lo ? y : cy[v] + y;
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s_map[0][w][lane * V + v] = cy[v];
            s_map[1][w][lane * V + v] = ch[v];
            s_map[2][w][lane * V + v] = decay(cy[v]);
        }
    }
    if (g > 0) __syncthreads();
    if (w == 0) {
        float cy[V], ch[V], in[V], P[V], cp[V];
#pragma unroll
        for (int v = 0; v < V; ++v) cy[v] = 0.0f, ch[v] = 0.0f, P[v] = decay(Y[v]);
#pragma unroll 1   // (two at a time spill registers in the backward)
        for (int k = 0; k * m < g; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                ch[v] = fmaf(s_map[2][k][lane * V + v], ch[v], s_map[1][k][lane * V + v]);
                cy[v] += s_map[0][k][lane * V + v];
            }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            cp[v] = decay(cy[v]);
            asm volatile("" : "+v"(cp[v]), "+v"(P[v]));   // (ready before the wait, which they would lengthen)
        }
        if (pos == g) {   // the first group: position 0 has taken the start in (0 elsewhere)
#pragma unroll
            for (int v = 0; v < V; ++v) in[v] = start[v];
        } else {
            const uint64_t *src = base + (pos - g - 1) * stride;
            for (;;) {
                bool all = true;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const uint64_t u = chain_read(src + v);
                    in[v] = __uint_as_float((uint32_t)u);
                    all = all && (uint32_t)(u >> 32) == __float_as_uint(1.0f);
                }
                if (__all(all || !act)) break;
                __builtin_amdgcn_s_sleep(1);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            in[v] = fmaf(cp[v], in[v], ch[v]);
            out[v] = fmaf(P[v], in[v], H[v]);
            if (act && !ends && g == group - 1) chain_put(own + v, 1.0f, out[v]);
            s_in[lane * V + v] = in[v];
        }
    }
    __syncthreads();
}

// The chain's step where every item waits for the one before it: the words are the states alone, four
// bytes each (all ones meaning that nothing is there yet; a NaN state is published as the usual one).
// Arguments and results as chain_step's.
template <int V>
__device__ __forceinline__ void chain_hand(uint32_t *base, int64_t stride, int pos, bool ends, bool act, int lane,
                                           int w, const float (&Y)[V], const float (&H)[V], const float (&start)[V],
                                           float (&s_in)[64 * V], float (&out)[V]) {
    if (w == 0) {
        float in[V], P[V];
        uint32_t *own = base + pos * stride;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = decay(Y[v]);
            asm volatile("" : "+v"(P[v]));   // (ready before the wait, which it would lengthen)
        }
        if (pos == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) in[v] = start[v];
        } else {
            for (;;) {
                bool all = true;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const uint32_t u = __hip_atomic_load(own - stride + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    in[v] = __uint_as_float(u);
                    all = all && u != kWordEmpty;
                }
                if (__all(all || !act)) break;
                __builtin_amdgcn_s_sleep(1);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            out[v] = fmaf(P[v], in[v], H[v]);
            if (act && !ends)
                __hip_atomic_store(own + v, out[v] != out[v] ? 0x7fc00000u : __float_as_uint(out[v]), __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            s_in[lane * V + v] = in[v];
        }
    }
    __syncthreads();
}

// Which item this workgroup takes: (sequence, tile, position along the chain), or pos < 0 for none.
// A queue's chains are walked together, position by position.  Chains are numbered sequence by
// sequence, or, where the sequences have lengths of their own, tile by tile, so that every queue gets
// its share of the long ones (B8 L2048 D5120 bf16 gated, lengths from 2048 down to 0: 134 us in the order of
// the sequences, 112 like this, backward 266 and 232).
struct GatedItem {
    int b, tile, pos;
};
// (32-bit unsigned: chains and items are below 2^23, and 64-bit divisions cost every wave's start.)
__device__ __forceinline__ GatedItem gated_item(uint32_t chains, uint32_t tiles, uint32_t nitem, bool ragged,
                                                int *counters, uint32_t queues, uint32_t run, int *slot) {
    const uint32_t turn = run == 1 ? blockIdx.x : blockIdx.x / kGatedRun, lane = run == 1 ? 0 : blockIdx.x % kGatedRun;
    const uint32_t round = turn / queues, q = turn - round * queues;
    const uint32_t first = chains * q / queues, nq = chains * (q + 1) / queues - first;
    if (nq == 0) return {0, 0, -1};
    uint32_t n = round * run + lane;
    if (counters) {   // (one item per sequence: no chain, any order will do)
        if (threadIdx.x == 0)
            *slot = __hip_atomic_fetch_add(&counters[q * kGatedCounterStride], 1, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        n = __builtin_amdgcn_readfirstlane(*slot);
    }
    if (n >= nq * nitem) return {0, 0, -1};
    const uint32_t pos = n / nq, chain = first + n - pos * nq;
    const uint32_t per = ragged ? chains / tiles : tiles, hi = chain / per, lo = chain - hi * per;
    return ragged ? GatedItem{(int)lo, (int)hi, (int)pos} : GatedItem{(int)hi, (int)lo, (int)pos};
}

// Fills the chain's words with ones (n 16-byte pairs of them: the array is padded) and clears the
// counters behind them.
static __global__ void __launch_bounds__(256)
gated_clear_kernel(u32x4_t *__restrict__ words, int64_t n, u32x4_t *__restrict__ counters) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const u32x4_t ones = {~0u, ~0u, ~0u, ~0u}, zeros = {0, 0, 0, 0};
    if (i < n) words[i] = ones;
    else if (i - n < kGatedQueues * kGatedCounterStride / 4) counters[i - n] = zeros;
}

// A token's coefficients for one channel.  STEP: the state goes from token to token by a alone.  (Between the
// chunks of a scan it goes by the sums of y; inside one, 64 or 128 tokens add up to 4e-7 on average, below the
// polynomial's own error for bf16, which therefore leaves the unit's value: B8 L2048 D5120 166 us, 167 to 170
// with 1 - u.)
struct GatedCoeff {
    float s, i, y, a, q;   // sigmoid(r), sigmoid(g), log2 a, a, 1 - a^2
};
template <typename IO, bool STEP = false>
__device__ __forceinline__ GatedCoeff gated_coeff(float r, float g, float a2) {
    GatedCoeff c;
    c.s = sigmoid_f32(r);
    c.i = sigmoid_f32(g);
    c.y = a2 * c.s;
    const float e = hw_exp2(c.y), u = one_minus<IO>(c.y, e);
    c.a = (STEP || sizeof(IO) == 4) && c.y > kNearOne<IO> ? 1.0f - u : e;
    c.q = fmaf(u, c.a, u);
    return c;
}

// OUT: y and last_state are written; otherwise only the states.  states: the state at the end
// of every kGatedChunk tokens but a sequence's last, for the backward pass (NULL where the words are that
// already, or there is one chunk).
// M: the tokens of an item in units of kGatedChunk.
template <typename IO, int V, int T, int K, bool OUT, bool NT>
__global__ void __launch_bounds__(64 * K)
gated_scan_kernel(const IO *__restrict__ x, const IO *__restrict__ r, const IO *__restrict__ g,
                  const float *__restrict__ A, const IO *__restrict__ z, const float *h0,
                  const int32_t *__restrict__ seq_lens, IO *__restrict__ y, float *last,
                  float *states, void *words, int *counters, int64_t L, int64_t D, int tiles, int chains, int nitem,
                  int nchunk, int queues, int run, int group) {
    constexpr int C = T * K, M = C / kGatedChunk;
    static_assert(K == kGatedWaves && C % kGatedChunk == 0 && K % M == 0, "a stored state is at a wave's end");
    using Row = row_words<V, IO, NT>;
    __shared__ float s_P[K][64 * V], s_Y[K][64 * V], s_H[K][64 * V], s_in[64 * V];
    __shared__ float s_map[3][kGatedWaves][64 * V];
    __shared__ int s_slot;
    const GatedItem it = gated_item(chains, tiles, nitem, seq_lens != nullptr, counters, queues, run, &s_slot);
    if (it.pos < 0) return;
    const int b = it.b, c = it.pos;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The lane's first channel.  Of an odd width the last lane takes the last V channels: those it
    // shares with its neighbour (a lane of this wave: the host sees to it) get the same values from both.
    const int64_t dl = (int64_t)it.tile * 64 * V + lane * V;
    const bool act = dl < D;
    const int64_t d = min(dl, D - V);
    const uint32_t lofs = (uint32_t)d * (uint32_t)sizeof(IO);
    const int64_t Lb = seq_lens ? min((int64_t)max(seq_lens[b], 0), L) : L;
    const int64_t t0 = (int64_t)c * C + w * T;
    const int64_t row0 = (int64_t)b * L;
    const int nlive = (int)((Lb + C - 1) / C);   // items of this sequence that hold tokens
    // the wave's tokens that exist, and those with inputs (none or fewer: t0 is past the end)
    const int nrow = (int)min((int64_t)T, L - t0), nin = (int)min((int64_t)T, Lb - t0);
    // Row k of the wave is at lofs + k * pitch from its first one, in 32 bits (dim is at most 2^26): an
    // addition for the row's accesses, whatever their number.
    const uint32_t pitch = (uint32_t)D * (uint32_t)sizeof(IO);
    const int64_t e0 = (row0 + t0) * D;

    if (c >= nlive) {   // past the sequence's end
        if constexpr (OUT) {
            if (act) {
                const float zero[V] = {};
                for (int k = 0; k < nrow; ++k) Row::store(y + e0, lofs + k * pitch, zero);
                if (last && c == 0 && w == 0)
                    for (int v = 0; v < V; ++v) last[(int64_t)b * D + d + v] = h0 ? h0[(int64_t)b * D + d + v] : 0.0f;
            }
        }
        return;
    }

    // every load of the wave first (rows past the end: the last row again)
    const int64_t ei = (row0 + min(t0, Lb - 1)) * D;
    const int klast = max(nin, 1) - 1;
    Row rr[T], rg[T], rx[T], rz[OUT ? T : 1];
#pragma unroll
    for (int k = 0; k < T; ++k) {
        const uint32_t ofs = lofs + min(k, klast) * pitch;
        rr[k].load(r + ei, ofs);
        rg[k].load(g + ei, ofs);
        rx[k].load(x + ei, ofs);
    }
    float a2[V];
#pragma unroll
    for (int v = 0; v < V; ++v) a2[v] = A[d + v] * kLog2e;

    // Tokens past the end become the identity (a = 1, an input of 0) without a test per value below.
    if (nin < T) {
#pragma unroll
        for (int k = 0; k < T; ++k)
            if (k >= nin) {
                rr[k].fill(minus_inf_words<IO>());
                rg[k].fill(0);
                rx[k].fill(0);
            }
    }

    // 1. the coefficients and the wave's map
    float a[T][V], bb[T][V], Y[V], H[V];
#pragma unroll
    for (int v = 0; v < V; ++v) Y[v] = 0.0f, H[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < T; ++k) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const GatedCoeff cf = gated_coeff<IO>(rr[k].get(v), rg[k].get(v), a2[v]);
            a[k][v] = cf.a;
            bb[k][v] = __builtin_amdgcn_sqrtf(cf.q) * cf.i * rx[k].get(v);
            Y[v] += cf.y;
            H[v] = fmaf(a[k][v], H[v], bb[k][v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s_P[w][lane * V + v] = hw_exp2(Y[v]);   // (inside the chunk, where nothing adds up, it will do)
        s_Y[w][lane * V + v] = Y[v];
        s_H[w][lane * V + v] = H[v];
    }
    // (the gate is requested here: it is needed last, and comes while the chain is waited for)
    if constexpr (OUT) {
        if (z) {
#pragma unroll
            for (int k = 0; k < T; ++k) rz[k].load(z + ei, lofs + min(k, klast) * pitch);
        }
    }
    __syncthreads();

    // 2. the chunk's map, the state at its start, the state at its end
    const bool ends = c == nlive - 1;
    float start[V] = {}, out[V];
    if (w == 0) {
#pragma unroll
        for (int k = 1; k < K; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                H[v] = fmaf(s_P[k][lane * V + v], H[v], s_H[k][lane * V + v]);
                Y[v] += s_Y[k][lane * V + v];
            }
        // (read before anything is published: the chain's last item may write last_state over it)
        if (c == 0 && h0) {
#pragma unroll
            for (int v = 0; v < V; ++v) start[v] = h0[(int64_t)b * D + d + v];
        }
    }
    const int64_t chain0 = (int64_t)b * nitem * D + d;
    if (group == 1)
        chain_hand<V>(static_cast<uint32_t *>(words) + chain0, D, c, ends, act, lane, w, Y, H, start, s_in, out);
    else
        chain_step<V>(static_cast<uint64_t *>(words) + chain0, D, c, group, ends, act, lane, w, Y, H, start, s_map,
                      s_in, out);
    float *st = states ? states + ((int64_t)b * nchunk + c * M) * D + d : nullptr;   // the item's states
    if (w == 0 && act) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (ends && OUT && last) last[(int64_t)b * D + d + v] = out[v];
            if (!ends && st) st[(M - 1) * D + v] = out[v];
        }
    }
    if constexpr (OUT || M > 1) {
        // 3. the state at the wave's start, and its tokens from there
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = s_in[lane * V + v];
        for (int k = 0; k < w; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(s_P[k][lane * V + v], h[v], s_H[k][lane * V + v]);
        if constexpr (M > 1) {   // the states inside the item
            const int j = w / (K / M);
            if (st && j > 0 && w % (K / M) == 0 && act && (int64_t)(c * M + j) * kGatedChunk < Lb) {
#pragma unroll
                for (int v = 0; v < V; ++v) st[(j - 1) * D + v] = h[v];
            }
        }
        if constexpr (OUT) {
#pragma unroll
            for (int k = 0; k < T; ++k) {
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    h[v] = fmaf(a[k][v], h[v], bb[k][v]);
                    o[v] = z ? h[v] * silu_f32(rz[k].get(v)) : h[v];
                    if (k >= nin) o[v] = 0.0f;
                }
                if (act && k < nrow) Row::store(y + e0, lofs + k * pitch, o);
            }
        }
    }
}

// The gradients.  lambda_t = dh_t + G_t with G_t = a_{t+1} lambda_{t+1}, dh_t = dy_t silu(z_t), is
// the same kind of recurrence run from the end (the map of a span is G -> P G + H' with the same
// P), so the items and the chain are the forward's in the other order; the states come from
// the array that the forward left (the state at the end of every chunk).  Each wave forms both maps of
// its tokens, then walks them forwards for the states and backwards for the gradients.  The
// coefficients that cost transcendentals (both sigmoids, the decay) stay in registers in between;
// 1 - a^2 is formed again.  dA's share of the item goes to part[item], summed afterwards in order.
template <typename IO, int V, bool GATE, bool NT>
__global__ void __launch_bounds__(64 * kGatedWaves)
__attribute__((amdgpu_waves_per_eu(4)))
gated_bwd_kernel(const IO *__restrict__ x, const IO *__restrict__ r, const IO *__restrict__ g,
                 const float *__restrict__ A, const IO *__restrict__ z, const float *__restrict__ h0,
                 const int32_t *__restrict__ seq_lens, const IO *__restrict__ dy, const float *__restrict__ dlast,
                 const float *__restrict__ states, IO *__restrict__ dx, IO *__restrict__ dr, IO *__restrict__ dg,
                 IO *__restrict__ dz, float *__restrict__ part, float *__restrict__ dh0, void *words,
                 int *counters, int64_t L, int64_t D, int tiles, int chains, int nchunk, int queues, int run,
                 int group) {
    constexpr int T = kGatedRows, K = kGatedWaves, C = kGatedChunk;
    using Row = row_words<V, IO, NT>;
    __shared__ float s_P[K][64 * V], s_Y[K][64 * V], s_H[K][64 * V], s_G[K][64 * V], s_in[64 * V];
    __shared__ float s_map[3][kGatedWaves][64 * V];
    __shared__ int s_slot;
    const GatedItem it = gated_item(chains, tiles, nchunk, seq_lens != nullptr, counters, queues, run, &s_slot);
    if (it.pos < 0) return;
    const int b = it.b, c = nchunk - 1 - it.pos;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t dl = (int64_t)it.tile * 64 * V + lane * V;
    const bool act = dl < D;
    const int64_t d = min(dl, D - V);
    const uint32_t lofs = (uint32_t)d * (uint32_t)sizeof(IO);
    const int64_t Lb = seq_lens ? min((int64_t)max(seq_lens[b], 0), L) : L;
    const int64_t t0 = (int64_t)c * C + w * T;
    const int64_t row0 = (int64_t)b * L;
    const int64_t ch = (int64_t)b * D + d;                      // the channel's place in [batch][dim]
    const int64_t item = ((int64_t)b * nchunk + c) * D + d;     // and in [batch][chunk][dim]
    const int nlive = (int)((Lb + C - 1) / C);
    const int nrow = (int)min((int64_t)T, L - t0), nin = (int)min((int64_t)T, Lb - t0);
    const uint32_t pitch = (uint32_t)D * (uint32_t)sizeof(IO);
    const int64_t e0 = (row0 + t0) * D;

    if (c >= nlive) {
        if (act) {
            const float zero[V] = {};
            for (int k = 0; k < nrow; ++k) {
                const uint32_t ofs = lofs + k * pitch;
                Row::store(dx + e0, ofs, zero);
                Row::store(dr + e0, ofs, zero);
                Row::store(dg + e0, ofs, zero);
                if constexpr (GATE) Row::store(dz + e0, ofs, zero);
            }
            if (w == 0)
                for (int v = 0; v < V; ++v) {
                    part[item + v] = 0.0f;
                    if (c == 0 && dh0) dh0[ch + v] = dlast ? dlast[ch + v] : 0.0f;
                }
        }
        return;
    }

    const int64_t ei = (row0 + min(t0, Lb - 1)) * D;
    const int klast = max(nin, 1) - 1;
    Row rr[T], rg[T], rx[T], ry[T], rz[GATE ? T : 1];
#pragma unroll
    for (int k = 0; k < T; ++k) {
        const uint32_t ofs = lofs + min(k, klast) * pitch;
        rr[k].load(r + ei, ofs);
        rg[k].load(g + ei, ofs);
        rx[k].load(x + ei, ofs);
        ry[k].load(dy + ei, ofs);
    }
    if constexpr (GATE) {
#pragma unroll
        for (int k = 0; k < T; ++k) rz[k].load(z + ei, lofs + min(k, klast) * pitch);
    }
    float Ad[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Ad[v] = A[d + v];
        // the state at the chunk's start
        h[v] = c == 0 ? (h0 ? h0[ch + v] : 0.0f) : states[item - D + v];
    }

    // Tokens past the end become the identity, and their gradients zero, without a test per value below.
    if (nin < T) {
#pragma unroll
        for (int k = 0; k < T; ++k)
            if (k >= nin) {
                rr[k].fill(minus_inf_words<IO>());
                rg[k].fill(0);
                rx[k].fill(0);
                ry[k].fill(0);
                if constexpr (GATE) rz[k].fill(0);
            }
    }

    // 1. the coefficients and the wave's two maps
    float s[T][V], i[T][V], a[T][V], bb[T][V], Y[V], H[V], G[V];
#pragma unroll
    for (int v = 0; v < V; ++v) Y[v] = 0.0f, H[v] = 0.0f, G[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < T; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const GatedCoeff cf = gated_coeff<IO>(rr[k].get(v), rg[k].get(v), Ad[v] * kLog2e);
            s[k][v] = cf.s;
            i[k][v] = cf.i;
            a[k][v] = cf.a;
            bb[k][v] = __builtin_amdgcn_sqrtf(cf.q) * cf.i * rx[k].get(v);
            Y[v] += cf.y;
            H[v] = fmaf(cf.a, H[v], bb[k][v]);
        }
    // dh_t, and with a gate the factor of h_t in dz: silu(z) = z sz, silu'(z) = sz (1 + z (1 - sz))
    auto grad_in = [&](int k, int v, float &dzh) {
        const float dyv = ry[k].get(v);
        if constexpr (!GATE) return dyv;
        const float zz = rz[GATE ? k : 0].get(v), sz = sigmoid_f32(zz), g = zz * sz;
        dzh = dyv * fmaf(g, 1.0f - sz, sz);
        return dyv * g;
    };
#pragma unroll
    for (int k = T - 1; k >= 0; --k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float dzh;
            G[v] = a[k][v] * (grad_in(k, v, dzh) + G[v]);
        }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s_P[w][lane * V + v] = hw_exp2(Y[v]);
        s_Y[w][lane * V + v] = Y[v];
        s_H[w][lane * V + v] = H[v];
        s_G[w][lane * V + v] = G[v];
    }
    __syncthreads();

    // 2. the adjoint at the chunk's end, and the one that it hands on
    const bool starts = c == nlive - 1;
    float start[V] = {}, out[V];
    if (w == 0) {   // the chunk's map (over Y and G, which wave 0 needs no more)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Y[v] = s_Y[K - 1][lane * V + v];
            G[v] = s_G[K - 1][lane * V + v];
        }
#pragma unroll
        for (int k = K - 2; k >= 0; --k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                G[v] = fmaf(s_P[k][lane * V + v], G[v], s_G[k][lane * V + v]);
                Y[v] += s_Y[k][lane * V + v];
            }
        if (starts && dlast) {
#pragma unroll
            for (int v = 0; v < V; ++v) start[v] = dlast[ch + v];
        }
    }
    const int64_t chain0 = ((int64_t)b * nchunk + nlive - 1) * D + d;
    if (group == 1)
        chain_hand<V>(static_cast<uint32_t *>(words) + chain0, -D, nlive - 1 - c, c == 0, act, lane, w, Y, G, start,
                      s_in, out);
    else
        chain_step<V>(static_cast<uint64_t *>(words) + chain0, -D, nlive - 1 - c, group, c == 0, act, lane, w, Y, G,
                      start, s_map, s_in, out);
    if (w == 0 && act && c == 0 && dh0) {
#pragma unroll
        for (int v = 0; v < V; ++v) dh0[ch + v] = out[v];
    }

    // 3. the states before the wave's tokens (over bb), the adjoint after its last, the gradients.
    // What follows is computed from the registers named here alone: without this the compiler keeps
    // what it derived from them above (1 - a^2, widened inputs), more registers than four waves
    // per SIMD leave a lane.
#pragma unroll
    for (int k = 0; k < T; ++k) {
        rx[k].opaque();
        ry[k].opaque();
        if constexpr (GATE) rz[k].opaque();
#pragma unroll
        for (int v = 0; v < V; ++v) asm volatile("" : "+v"(s[k][v]), "+v"(i[k][v]), "+v"(a[k][v]));
    }
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
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float dzh = 0.0f;
            const float lam = grad_in(k, v, dzh) + G[v];
            if constexpr (GATE) oz[v] = dzh * hT[v];
            G[v] = a[k][v] * lam;
            const float u = one_minus<IO>(Ad[v] * kLog2e * s[k][v], a[k][v]), q = fmaf(u, a[k][v], u);
            // 1 / beta; where 1 - a^2 is zero (or below what the unit resolves) the terms with it are dropped
            const float rb = fabsf(q) < FLT_MIN ? 0.0f : __builtin_amdgcn_rsqf(q);
            ox[v] = lam * (q * rb) * i[k][v];            // lambda beta i
            const float t = ox[v] * rx[k].get(v);        // lambda beta i x
            og[v] = fmaf(-t, i[k][v], t);
            const float e = a[k][v] * rb;                // i x a^2 / beta = beta i x (a / beta)^2
            const float ds = fmaf(-t, e * e, G[v] * bb[k][v]) * s[k][v];
            dA[v] += ds;
            orr[v] = ds * fmaf(-Ad[v], s[k][v], Ad[v]);
            hT[v] = bb[k][v];
        }
        if (act && k < nrow) {
            const uint32_t ofs = lofs + k * pitch;
            Row::store(dx + e0, ofs, ox);
            Row::store(dr + e0, ofs, orr);
            Row::store(dg + e0, ofs, og);
            if constexpr (GATE) Row::store(dz + e0, ofs, oz);
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

// out[d] = sum of the n rows of part, in an order of their own: kColumnGroups groups of threads take
// every kColumnGroups-th row of kColumnCols columns, and their sums are added in order.  Bound: the
// latency of a few dependent loads (64 rows of 1536 columns: 4.3 us).
constexpr int kColumnCols = 32, kColumnGroups = 32;
static __global__ void __launch_bounds__(kColumnCols * kColumnGroups)
column_sum_kernel(const float *__restrict__ part, float *__restrict__ out, int64_t n, int64_t D) {
    __shared__ float red[kColumnGroups][kColumnCols];
    const int col = threadIdx.x % kColumnCols, g = threadIdx.x / kColumnCols;
    const int64_t d = (int64_t)blockIdx.x * kColumnCols + col;
    float s = 0.0f;
    if (d < D)
#pragma unroll 8
        for (int64_t k = g; k < n; k += kColumnGroups) s += part[k * D + d];
    red[g][col] = s;
    __syncthreads();
    if (g == 0 && d < D) {
#pragma unroll
        for (int k = 1; k < kColumnGroups; ++k) s += red[k][col];
        out[d] = s;
    }
}

// One token of every sequence, the state updated in place.  The tensors are walked as flat arrays,
// kStepVec neighbouring elements per thread (they may lie in two rows; A's index wraps with them).
// Bound: HBM, 8 bytes of state and 4 or 5 I/O elements per channel (S256 D5120 bf16 with its gate:
// 23.6 MB, 5.3 us on the device).  The state is left in the caches for the next token.
constexpr int kStepVec = 4;
template <typename IO>
__global__ void __launch_bounds__(256)
gated_step_kernel(float *__restrict__ state, const IO *__restrict__ x, const IO *__restrict__ r,
                  const IO *__restrict__ g, const float *__restrict__ A, const IO *__restrict__ z,
                  IO *__restrict__ y, int64_t n, int64_t D) {
    typedef float any_f32 __attribute__((ext_vector_type(kStepVec), aligned(sizeof(float))));
    const int64_t base = (int64_t)blockIdx.x * (256 * kStepVec);
    const int64_t e = base + threadIdx.x * kStepVec;
    if (e >= n) return;
    auto token = [&](float rr, float gg, float xx, float Av, float h) {
        const GatedCoeff cf = gated_coeff<IO, true>(rr, gg, Av * kLog2e);
        return fmaf(cf.a, h, __builtin_amdgcn_sqrtf(cf.q) * cf.i * xx);
    };
    const int64_t d = e % D;
    if (e + kStepVec > n) {   // the array's last elements
        for (int64_t k = e; k < n; ++k) {
            const float h = token(io<IO>::ld(r, k), io<IO>::ld(g, k), io<IO>::ld(x, k), A[k % D], state[k]);
            state[k] = h;
            io<IO>::st(y, k, z ? h * silu_f32(io<IO>::ld(z, k)) : h);
        }
        return;
    }
    const uint32_t lofs = threadIdx.x * kStepVec * (uint32_t)sizeof(IO);
    row_words<kStepVec, IO> rr, rg, rx, rz;
    rr.load(r + base, lofs);
    rg.load(g + base, lofs);
    rx.load(x + base, lofs);
    if (z) rz.load(z + base, lofs);
    any_f32 h = *reinterpret_cast<const any_f32 *>(state + e), Av;
    if (d + kStepVec <= D) {
        Av = *reinterpret_cast<const any_f32 *>(A + d);
    } else {
#pragma unroll
        for (int k = 0; k < kStepVec; ++k) Av[k] = A[(d + k) % D];
    }
    float o[kStepVec];
#pragma unroll
    for (int k = 0; k < kStepVec; ++k) {
        h[k] = token(rr.get(k), rg.get(k), rx.get(k), Av[k], h[k]);
        o[k] = z ? h[k] * silu_f32(rz.get(k)) : h[k];
    }
    *reinterpret_cast<any_f32 *>(state + e) = h;
    row_words<kStepVec, IO>::store(y + base, lofs, o);
}

}  // namespace ssm
