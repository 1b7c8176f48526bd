// The gated linear recurrence's entry points (include/ssmscan.h): validation and launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gated_kernel.h"
#include "host_util.h"

namespace {

using namespace ssmlib;

constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr int64_t kMaxElems = int64_t(1) << 46;

// Sizes of the recurrence (dstate and chunk_len do not apply).
int check_gated_dims(const ssm_dims *dm, bool seq) {
    if (!dm) return fail(SSM_ERR_NULL, "dims is NULL");
    if (dm->batch < 0 || dm->dim < 0 || (seq && dm->seqlen < 0))
        return fail(SSM_ERR_SHAPE, "negative size (batch=%lld seqlen=%lld dim=%lld)", (long long)dm->batch,
                    (long long)dm->seqlen, (long long)dm->dim);
    if (dm->io_dtype != SSM_IO_F32 && dm->io_dtype != SSM_IO_BF16)
        return fail(SSM_ERR_DTYPE, "io_dtype %d is not SSM_IO_F32 (0) or SSM_IO_BF16 (1)", dm->io_dtype);
    if (dm->dim > kMaxDim / 16 || dm->batch > kMaxDim)   // (the column sums launch 32 threads per column)
        return fail(SSM_ERR_SHAPE, "dim larger than 2^26 or batch larger than 2^30");
    if (dm->batch > 0 && dm->dim > (int64_t(1) << 33) / dm->batch)
        return fail(SSM_ERR_SHAPE, "batch*dim exceeds 2^33 (grid size)");
    if (seq && (dm->seqlen > kMaxDim ||
                (dm->batch > 0 && dm->dim > 0 && dm->seqlen > kMaxElems / dm->batch / dm->dim)))
        return fail(SSM_ERR_SHAPE, "seqlen exceeds 2^30 or batch*seqlen*dim exceeds 2^46 elements");
    return SSM_OK;
}

size_t elem_size(const ssm_dims *dm) { return dm->io_dtype == SSM_IO_BF16 ? 2 : 4; }

int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    return ok();
}

// How the sequences are cut, and the workspace: the states [batch][nchunk][dim] that the backward
// starts from, then the chain's words [batch][items per sequence][dim] and the counters; one chunk per
// sequence needs none of it.
struct Plan {
    int64_t nchunk, tiles, chains, cells;
    int V;
    bool lines;   // rows start on 128-byte lines (of tensors that do)
    size_t state_bytes, word_bytes, bytes;
};
constexpr int64_t kCounterInts = ssm::kGatedQueues * ssm::kGatedCounterStride;

// Channels per lane: two bf16 or one fp32, four bytes an access; one bf16 too where tiles of two would
// leave CUs idle (at most one workgroup each: B1 L512 D2048, 128 items: 7.4 against 9.8 us, backward 10.1
// against 12.9; B1 L4096 D256: 9.0 and 11.7, 11.8 and 15.3), and where the last of an odd width's
// channels would be a tile of its own: its lane shares a channel with its neighbour, which has to be in
// the same wave, as a state that is advanced in place is read by one and written by the other.
int lane_channels(const ssm_dims *dm, int64_t nchunk) {
    if (dm->io_dtype != SSM_IO_BF16 || dm->dim % 128 == 1) return 1;
    return dm->batch * ((dm->dim + 127) / 128) * nchunk > 256 ? 2 : 1;
}

Plan make_plan(const ssm_dims *dm) {
    Plan p;
    p.nchunk = std::max<int64_t>((dm->seqlen + ssm::kGatedChunk - 1) / ssm::kGatedChunk, 1);
    p.V = lane_channels(dm, p.nchunk);
    p.lines = dm->dim * (int64_t)elem_size(dm) % 128 == 0;
    p.tiles = (dm->dim + 64 * p.V - 1) / (64 * p.V);
    p.chains = dm->batch * p.tiles;
    p.cells = dm->batch * p.nchunk * dm->dim;
    p.state_bytes = p.nchunk > 1 ? align256((size_t)p.cells * sizeof(float)) : 0;
    p.word_bytes = p.nchunk > 1 ? align256((size_t)p.cells * sizeof(uint64_t)) : 0;
    p.bytes = p.nchunk > 1 ? p.state_bytes + p.word_bytes + kCounterInts * sizeof(int) : 0;
    return p;
}

// Queues that share the chains (see the kernel): as many as there are XCDs, unless some would then be
// much longer than the average; every queue has as many workgroups as the longest needs, those without
// an item still have to be dispatched, and an XCD whose queue is done has nothing left.  Short chains,
// where hand-overs count, take a quarter more (B6 L1000 D1700 bf16, 84 chains: 29 us with eight queues, 31
// with seven, backward 53 and 59), long ones a thirty-second (B3 L10000 D772, 21 chains: 83 us with eight, 73
// with seven, backward 148 and 123; B1 L30000 D2900, 23 chains: 224 with eight, 213 with one, 436 and 407; B1
// L65536 D64, one chain: 146 with eight, 35 with one).
int queues_of(const Plan &p) {
    auto slots = [&](int64_t q) { return (p.chains + q - 1) / q * q; };
    int best = ssm::kGatedQueues;
    if (p.nchunk < 32 ? 4 * slots(best) <= 5 * p.chains : 32 * slots(best) <= 33 * p.chains) return best;
    for (int q = best - 1; q >= 1; --q)
        if (slots(q) < slots(best)) best = q;
    return best;
}

// Consecutive workgroups that draw from one queue: 1 where the launch is short (B2 L2048 D1536 fp32: 25 us
// with either, its backward 38.0 with 1, 38.4 with 8) or neighbouring tiles share lines; 8 where it is many
// rounds of the chip and rows are whole lines (B1 L131072 D2048 bf16, 16 chains: 534 us with 1, 475 with 8; B8
// L2048 D5120, 320 chains: 165 with either), or an XCD would have so few tiles that there is little to share
// (B1 L131072 D2047, 16 chains: 720 with 1, 628 with 8, backward 1,453 and 1,305; B2 L65536 D1500, 24 chains:
// 498 and 470, 991 and 962; but B8 L2048 D5119, 320 chains: 199 and 233, 368 and 429).
int run_of(const Plan &p, int64_t nitem) {
    return (p.lines || p.chains <= 32) && p.chains * nitem >= 4096 ? ssm::kGatedRun : 1;
}

// Items of a chain that share a hand-over (see the kernel), a power of two.  A hand-over takes about 1.2
// us, and while it runs every chain moves 0.013 us of data per item: with many chains every item can wait
// for the one before it, and the maps' traffic is saved (B8 L2048 D5120 bf16, 320 chains: 166 us with
// groups of one, 176 with eight, backward 303 and 313; B2 L8192 D5120, 80 chains: backward 301 with one,
// 308 with four), with few the hand-overs have to be shared (B1 L131072 D2048, 16 chains: 704 us with one,
// 482 with four, 475 with eight; B1 L65536 D512, 4 chains: 167 with two, 92 with eight, 86 with 16 or 32; D64,
// 1 chain: 98 with eight, 35 with 64; B2 L2048 D1536 fp32, 48 chains: 28 with one, 25 with two or four).
int group_of(const Plan &p) {
    int g = 1;
    if (p.chains < 64)
        while (g < ssm::kGatedGroup && g * p.chains < 96) g *= 2;
    return g;
}

// One workgroup per (chain, item), the chains dealt to the queues in turn.
int64_t grid_of(const Plan &p, int64_t nitem) {
    const int64_t q = queues_of(p), per = (p.chains + q - 1) / q * nitem, run = run_of(p, nitem);
    return (per + run - 1) / run * run * q;   // (per: items of the longest queue)
}

// A launch holds fewer than 2^32 threads.
int check_items(const Plan &p) {
    constexpr int64_t most = ((int64_t(1) << 32) - 1) / (64 * ssm::kGatedWaves);
    if (p.chains > most || grid_of(p, p.nchunk) > most)
        return fail(SSM_ERR_SHAPE, "batch * ceil(dim / %d) * ceil(seqlen / %d) exceeds 2^23 work items", 64 * p.V,
                    ssm::kGatedChunk);
    return SSM_OK;
}

// The chain's words, made ready for nitem items per sequence, and the counters at the workspace's end;
// returns the counters, NULL where there is no chain.
int *launch_clear(const Plan &p, void *words, void *ws, int64_t nitem, const ssm_dims *dm, hipStream_t st) {
    if (nitem == 1) return nullptr;
    ssm::u32x4_t *counters = reinterpret_cast<ssm::u32x4_t *>(static_cast<char *>(ws) + p.state_bytes + p.word_bytes);
    const int64_t bytes = dm->batch * nitem * dm->dim * (group_of(p) == 1 ? 4 : 8), n = (bytes + 15) / 16;
    hipLaunchKernelGGL(ssm::gated_clear_kernel, dim3((unsigned)((n + kCounterInts / 4 + 255) / 256)), dim3(256), 0, st,
                       static_cast<ssm::u32x4_t *>(words), n, counters);
    return reinterpret_cast<int *>(counters);
}

// Items of two chunks halve the hand-overs of a chain, at two workgroups per CU instead of three.  They
// pay where chains are long, as long as the halved number of items still fills the chip (B1 L131072 D2048
// bf16 gated: 563 us with one, 474 with two; B2 L8192 D3000: 146 and 126; B2 L8192 D2048 fp32: 132 and 116; but
// B3 L4096 D1400, 2112 chunks in all: 55 and 57).  Chains of 32 chunks gain in bf16 and lose in fp32, so that
// the rule leaves them (B8 L2048 D5120: 166 and 155, fp32 291 and 308).
int fwd_item_chunks(const ssm_dims *dm, const Plan &p) {
    const bool one_bf16 = dm->io_dtype == SSM_IO_BF16 && p.V == 1;   // (narrow or few: short chains, or few items)
    return !one_bf16 && p.nchunk >= 64 && p.chains * p.nchunk >= 2304 ? 2 : 1;
}

template <typename IO, int V, int T, int K, bool OUT, bool NT>
void launch_fwd_v(const void *x, const void *r, const void *g, const float *A, const void *z, const float *h0,
                  const int32_t *sl, void *y, float *last, void *ws, const ssm_dims *dm, const Plan &p,
                  hipStream_t st) {
    constexpr int64_t M = T * K / ssm::kGatedChunk;
    const int64_t nitem = (p.nchunk + M - 1) / M;
    // (with groups of one and an item per state the words are the states)
    const bool own = M > 1 || group_of(p) > 1;
    float *states = p.nchunk > 1 && own ? static_cast<float *>(ws) : nullptr;
    void *words = own ? static_cast<char *>(ws) + p.state_bytes : ws;
    int *counters = launch_clear(p, words, ws, nitem, dm, st);
    hipLaunchKernelGGL((ssm::gated_scan_kernel<IO, V, T, K, OUT, NT>), dim3((unsigned)grid_of(p, nitem)), dim3(64 * K),
                       0, st, static_cast<const IO *>(x), static_cast<const IO *>(r),
                       static_cast<const IO *>(g), A, static_cast<const IO *>(z), h0, sl, static_cast<IO *>(y), last,
                       states, words, counters, dm->seqlen, dm->dim, (int)p.tiles, (int)p.chains, (int)nitem,
                       (int)p.nchunk, queues_of(p), run_of(p, nitem), group_of(p));
}

template <bool OUT, bool NT>
void launch_fwd_n(const void *x, const void *r, const void *g, const float *A, const void *z, const float *h0,
                const int32_t *sl, void *y, float *last, void *ws, const ssm_dims *dm, const Plan &p,
                hipStream_t st) {
    const bool wide = fwd_item_chunks(dm, p) == 2;
    auto launch = dm->io_dtype == SSM_IO_F32
                      ? (wide ? launch_fwd_v<float, 1, 16, 8, OUT, NT> : launch_fwd_v<float, 1, 8, 8, OUT, NT>)
                  : p.V == 2 ? (wide ? launch_fwd_v<uint16_t, 2, 16, 8, OUT, NT>
                                     : launch_fwd_v<uint16_t, 2, 8, 8, OUT, NT>)
                             : launch_fwd_v<uint16_t, 1, 8, 8, OUT, NT>;
    launch(x, r, g, A, z, h0, sl, y, last, ws, dm, p, st);
}

template <bool OUT>
void launch_fwd(const void *x, const void *r, const void *g, const float *A, const void *z, const float *h0,
                const int32_t *sl, void *y, float *last, void *ws, const ssm_dims *dm, const Plan &p,
                hipStream_t st) {
    if (p.lines) launch_fwd_n<OUT, true>(x, r, g, A, z, h0, sl, y, last, ws, dm, p, st);
    else launch_fwd_n<OUT, false>(x, r, g, A, z, h0, sl, y, last, ws, dm, p, st);
}

// The backward's workspace: the forward's (its states, where no checkpoints are given; its chain is the
// backward's afterwards), and dA's shares [batch][nchunk][dim].
size_t bwd_bytes(const ssm_dims *dm, const Plan &p) {
    if (dm->batch == 0 || dm->dim == 0) return 0;
    return p.bytes + align256((size_t)p.cells * sizeof(float));
}

template <typename IO, int V>
void launch_bwd_v(const void *x, const void *r, const void *g, const float *A, const void *z, const float *h0,
                  const int32_t *sl, const void *dy, const float *dlast, const void *states, void *dx, void *dr,
                  void *dg, void *dz, float *part, float *dh0, void *ws, const ssm_dims *dm, const Plan &p,
                  hipStream_t st) {
    void *words = static_cast<char *>(ws) + p.state_bytes;
    int *counters = launch_clear(p, words, ws, p.nchunk, dm, st);
    auto kern = z ? (p.lines ? ssm::gated_bwd_kernel<IO, V, true, true> : ssm::gated_bwd_kernel<IO, V, true, false>)
                  : (p.lines ? ssm::gated_bwd_kernel<IO, V, false, true> : ssm::gated_bwd_kernel<IO, V, false, false>);
    hipLaunchKernelGGL(kern, dim3((unsigned)grid_of(p, p.nchunk)), dim3(64 * ssm::kGatedWaves), 0, st,
                       static_cast<const IO *>(x), static_cast<const IO *>(r), static_cast<const IO *>(g), A,
                       static_cast<const IO *>(z), h0, sl, static_cast<const IO *>(dy), dlast,
                       static_cast<const float *>(states), static_cast<IO *>(dx), static_cast<IO *>(dr),
                       static_cast<IO *>(dg), static_cast<IO *>(dz), part, dh0, words, counters, dm->seqlen, dm->dim,
                       (int)p.tiles, (int)p.chains, (int)p.nchunk, queues_of(p), run_of(p, p.nchunk), group_of(p));
}

}  // namespace

extern "C" {

size_t ssm_gated_scan_workspace_bytes(const ssm_dims *dims) {
    if (check_gated_dims(dims, true) != SSM_OK || dims->batch == 0 || dims->dim == 0) return 0;
    const Plan p = make_plan(dims);
    return check_items(p) == SSM_OK ? p.bytes : 0;
}

int ssm_gated_scan_plan(const ssm_dims *dims, int backward, ssm_gated_plan *out) {
    if (!out) return fail(SSM_ERR_NULL, "out is NULL");
    *out = {};
    const int rc = check_gated_dims(dims, true);
    if (rc != SSM_OK) return rc;
    if (dims->batch == 0 || dims->dim == 0) return ok();
    const Plan p = make_plan(dims);
    if (const int e = check_items(p)) return e;
    out->item_chunks = backward ? 1 : fwd_item_chunks(dims, p);
    const int64_t nitem = (p.nchunk + out->item_chunks - 1) / out->item_chunks;
    out->chains = p.chains;
    out->items = nitem;
    out->workgroups = grid_of(p, nitem);
    out->lane_channels = p.V;
    out->group = group_of(p);
    out->queues = queues_of(p);
    out->run = run_of(p, nitem);
    return ok();
}

size_t ssm_gated_scan_bwd_workspace_bytes(const ssm_dims *dims) {
    if (check_gated_dims(dims, true) != SSM_OK || dims->batch == 0 || dims->dim == 0) return 0;
    const Plan p = make_plan(dims);
    return check_items(p) == SSM_OK ? bwd_bytes(dims, p) : 0;
}

int ssm_gated_scan_fwd(const void *x, const void *r, const void *g, const float *A, const void *z,
                       const float *initial_state, const int32_t *seq_lens, void *y, float *last_state,
                       const ssm_dims *dims, void *workspace, size_t workspace_bytes, void *stream) {
    const int rc = check_gated_dims(dims, true);
    if (rc != SSM_OK) return rc;
    const size_t es = elem_size(dims);
    if (!aligned(x, es) || !aligned(r, es) || !aligned(g, es) || !aligned(z, es) || !aligned(y, es) ||
        !aligned(A, 4) || !aligned(initial_state, 4) || !aligned(seq_lens, 4) || !aligned(last_state, 4))
        return fail(SSM_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    if (dims->batch == 0 || dims->dim == 0) return ok();
    if (!A || (dims->seqlen > 0 && (!x || !r || !g || !y)))
        return fail(SSM_ERR_NULL, "required pointer is NULL (x=%p r=%p g=%p A=%p y=%p)", x, r, g, (const void *)A, y);
    const Plan p = make_plan(dims);
    if (const int e = check_items(p)) return e;
    if (p.bytes > 0 && !workspace) return fail(SSM_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", p.bytes);
    if (workspace_bytes < p.bytes)
        return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes,
                    p.bytes);
    if (p.bytes > 0 && !aligned(workspace, 16)) return fail(SSM_ERR_ALIGN, "workspace not 16-byte aligned");
    launch_fwd<true>(x, r, g, A, z, initial_state, seq_lens, y, last_state, workspace, dims, p,
                     static_cast<hipStream_t>(stream));
    return launched();
}

int ssm_gated_scan_bwd(const void *x, const void *r, const void *g, const float *A, const void *z,
                       const float *initial_state, const int32_t *seq_lens, const void *dy, const float *dlast_state,
                       const void *checkpoints, size_t checkpoints_bytes, void *dx, void *dr, void *dg, float *dA,
                       void *dz, float *dinitial_state, const ssm_dims *dims, void *workspace, size_t workspace_bytes,
                       void *stream) {
    const int rc = check_gated_dims(dims, true);
    if (rc != SSM_OK) return rc;
    const size_t es = elem_size(dims);
    if (!aligned(x, es) || !aligned(r, es) || !aligned(g, es) || !aligned(z, es) || !aligned(dy, es) ||
        !aligned(dx, es) || !aligned(dr, es) || !aligned(dg, es) || !aligned(dz, es) || !aligned(A, 4) ||
        !aligned(dA, 4) || !aligned(initial_state, 4) || !aligned(seq_lens, 4) || !aligned(dlast_state, 4) ||
        !aligned(dinitial_state, 4))
        return fail(SSM_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    if (dims->dim == 0) return ok();
    if (!dA) return fail(SSM_ERR_NULL, "dA is NULL");
    const Plan p = make_plan(dims);
    if (dims->batch > 0) {
        if (!A || (dims->seqlen > 0 && (!x || !r || !g || !dy || !dx || !dr || !dg)))
            return fail(SSM_ERR_NULL, "required pointer is NULL");
        if (dims->seqlen > 0 && z && !dz) return fail(SSM_ERR_NULL, "z is given but dz is NULL");
        if (const int e = check_items(p)) return e;
        const size_t need = bwd_bytes(dims, p);
        if (!workspace) return fail(SSM_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
        if (workspace_bytes < need)
            return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes,
                        need);
        if (checkpoints && checkpoints_bytes < p.bytes)
            return fail(SSM_ERR_WORKSPACE, "checkpoints of %zu bytes are smaller than the %zu needed",
                        checkpoints_bytes, p.bytes);
        if (!aligned(workspace, 16) || !aligned(checkpoints, 16))
            return fail(SSM_ERR_ALIGN, "workspace or checkpoints not 16-byte aligned");
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    float *part = reinterpret_cast<float *>(ws + p.bytes);
    if (dims->batch > 0) {
        const void *states = checkpoints ? checkpoints : workspace;
        if (!checkpoints && p.nchunk > 1)   // (a single chunk starts from the initial state)
            launch_fwd<false>(x, r, g, A, nullptr, initial_state, seq_lens, nullptr, nullptr, workspace, dims, p, st);
        auto bwd = dims->io_dtype == SSM_IO_F32 ? launch_bwd_v<float, 1>
                   : p.V == 2                   ? launch_bwd_v<uint16_t, 2>
                                                : launch_bwd_v<uint16_t, 1>;
        bwd(x, r, g, A, z, initial_state, seq_lens, dy, dlast_state, states, dx, dr, dg, dz, part, dinitial_state,
            ws, dims, p, st);
    }
    hipLaunchKernelGGL(ssm::column_sum_kernel,
                       dim3((unsigned)((dims->dim + ssm::kColumnCols - 1) / ssm::kColumnCols)),
                       dim3(ssm::kColumnCols * ssm::kColumnGroups), 0, st, part, dA, dims->batch * p.nchunk, dims->dim);
    return launched();
}

int ssm_gated_step(float *state, const void *x, const void *r, const void *g, const float *A, const void *z, void *y,
                   const ssm_dims *dims, void *stream) {
    const int rc = check_gated_dims(dims, false);
    if (rc != SSM_OK) return rc;
    const size_t es = elem_size(dims);
    if (!aligned(state, 4) || !aligned(x, es) || !aligned(r, es) || !aligned(g, es) || !aligned(A, 4) ||
        !aligned(z, es) || !aligned(y, es))
        return fail(SSM_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    if (dims->batch == 0 || dims->dim == 0) return ok();
    if (!state || !x || !r || !g || !A || !y) return fail(SSM_ERR_NULL, "required pointer is NULL");
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t n = dims->batch * dims->dim;
    const dim3 grid((unsigned)((n + 256 * ssm::kStepVec - 1) / (256 * ssm::kStepVec)));
    if (es == 2)
        hipLaunchKernelGGL(ssm::gated_step_kernel<uint16_t>, grid, dim3(256), 0, st, state,
                           static_cast<const uint16_t *>(x), static_cast<const uint16_t *>(r),
                           static_cast<const uint16_t *>(g), A, static_cast<const uint16_t *>(z),
                           static_cast<uint16_t *>(y), n, dims->dim);
    else
        hipLaunchKernelGGL(ssm::gated_step_kernel<float>, grid, dim3(256), 0, st, state,
                           static_cast<const float *>(x), static_cast<const float *>(r),
                           static_cast<const float *>(g), A, static_cast<const float *>(z), static_cast<float *>(y),
                           n, dims->dim);
    return launched();
}

}  // extern "C"
