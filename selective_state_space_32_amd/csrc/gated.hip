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
    if (dm->dim > kMaxDim || dm->batch > kMaxDim) return fail(SSM_ERR_SHAPE, "dim or batch larger than 2^30");
    if (dm->batch > 0 && dm->dim > (int64_t(1) << 36) / dm->batch)
        return fail(SSM_ERR_SHAPE, "batch*dim exceeds 2^36 (grid size)");
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

// How the sequences are cut, and the workspace: the chain's words [batch][nchunk][dim], then the
// counters; one chunk per sequence needs neither.
struct Plan {
    int64_t nchunk, tiles, chains, words;
    int V;
    size_t word_bytes, bytes;
};
constexpr size_t kCounterBytes = sizeof(int) * ssm::kGatedGroups * ssm::kGatedCounterStride;

Plan make_plan(const ssm_dims *dm) {
    Plan p;
    p.V = dm->dim >= 2 ? 2 : 1;
    p.nchunk = std::max<int64_t>((dm->seqlen + ssm::kGatedChunk - 1) / ssm::kGatedChunk, 1);
    p.tiles = (dm->dim + 64 * p.V - 1) / (64 * p.V);
    p.chains = dm->batch * p.tiles;
    p.words = dm->batch * p.nchunk * dm->dim;
    p.word_bytes = p.nchunk > 1 ? align256((size_t)p.words * sizeof(uint64_t)) : 0;
    p.bytes = p.nchunk > 1 ? p.word_bytes + kCounterBytes : 0;
    return p;
}

// One workgroup per (chain, chunk), the chains dealt to the groups in turn.
int64_t items(const Plan &p) {
    return (p.chains + ssm::kGatedGroups - 1) / ssm::kGatedGroups * ssm::kGatedGroups * p.nchunk;
}

int check_items(const Plan &p) {
    if (items(p) > (int64_t(1) << 31) - 1 || p.chains > (int64_t(1) << 31) - 1)
        return fail(SSM_ERR_SHAPE, "batch * ceil(dim / %d) * ceil(seqlen / %d) exceeds 2^31 work items", 64 * p.V,
                    ssm::kGatedChunk);
    return SSM_OK;
}

int *counters_of(const Plan &p, void *ws) {
    return p.nchunk > 1 ? reinterpret_cast<int *>(static_cast<char *>(ws) + p.word_bytes) : nullptr;
}

void launch_clear(const Plan &p, void *ws, hipStream_t st) {
    if (p.nchunk == 1) return;
    const int64_t n = p.words + ssm::kGatedGroups * ssm::kGatedCounterStride;
    hipLaunchKernelGGL(ssm::gated_clear_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st,
                       static_cast<uint64_t *>(ws), p.words, counters_of(p, ws));
}

template <typename IO, int V, bool OUT>
void launch_fwd_v(const void *x, const void *r, const void *g, const float *A, const void *z, const float *h0,
                  const int32_t *sl, void *y, float *last, void *ws, const ssm_dims *dm, const Plan &p,
                  hipStream_t st) {
    launch_clear(p, ws, st);
    hipLaunchKernelGGL((ssm::gated_scan_kernel<IO, V, OUT>), dim3((unsigned)items(p)), dim3(64 * ssm::kGatedWaves), 0,
                       st, static_cast<const IO *>(x), static_cast<const IO *>(r), static_cast<const IO *>(g), A,
                       static_cast<const IO *>(z), h0, sl, static_cast<IO *>(y), last, static_cast<uint64_t *>(ws),
                       counters_of(p, ws), dm->seqlen, dm->dim, (int)p.tiles, (int)p.chains, (int)p.nchunk);
}

template <bool OUT>
void launch_fwd(const void *x, const void *r, const void *g, const float *A, const void *z, const float *h0,
                const int32_t *sl, void *y, float *last, void *ws, const ssm_dims *dm, const Plan &p,
                hipStream_t st) {
    if (dm->io_dtype == SSM_IO_BF16) {
        if (p.V == 2) launch_fwd_v<uint16_t, 2, OUT>(x, r, g, A, z, h0, sl, y, last, ws, dm, p, st);
        else launch_fwd_v<uint16_t, 1, OUT>(x, r, g, A, z, h0, sl, y, last, ws, dm, p, st);
    } else {
        if (p.V == 2) launch_fwd_v<float, 2, OUT>(x, r, g, A, z, h0, sl, y, last, ws, dm, p, st);
        else launch_fwd_v<float, 1, OUT>(x, r, g, A, z, h0, sl, y, last, ws, dm, p, st);
    }
}

// The backward's workspace: the forward's (used where no checkpoints are given), its own chain, and
// dA's shares [batch][nchunk][dim].
size_t bwd_bytes(const ssm_dims *dm, const Plan &p) {
    if (dm->batch == 0 || dm->dim == 0) return 0;
    return 2 * p.bytes + align256((size_t)p.words * sizeof(float));
}

template <typename IO, int V>
void launch_bwd_v(const void *x, const void *r, const void *g, const float *A, const void *z, const float *h0,
                  const int32_t *sl, const void *dy, const float *dlast, const void *states, void *dx, void *dr,
                  void *dg, void *dz, float *part, float *dh0, void *ws, const ssm_dims *dm, const Plan &p,
                  hipStream_t st) {
    launch_clear(p, ws, st);
    hipLaunchKernelGGL((ssm::gated_bwd_kernel<IO, V>), dim3((unsigned)items(p)), dim3(64 * ssm::kGatedWaves), 0, st,
                       static_cast<const IO *>(x), static_cast<const IO *>(r), static_cast<const IO *>(g), A,
                       static_cast<const IO *>(z), h0, sl, static_cast<const IO *>(dy), dlast,
                       static_cast<const uint64_t *>(states), static_cast<IO *>(dx), static_cast<IO *>(dr),
                       static_cast<IO *>(dg), static_cast<IO *>(dz), part, dh0, static_cast<uint64_t *>(ws),
                       counters_of(p, ws), dm->seqlen, dm->dim, (int)p.tiles, (int)p.chains, (int)p.nchunk);
}

}  // namespace

extern "C" {

size_t ssm_gated_scan_workspace_bytes(const ssm_dims *dims) {
    if (check_gated_dims(dims, true) != SSM_OK || dims->batch == 0 || dims->dim == 0) return 0;
    const Plan p = make_plan(dims);
    return check_items(p) == SSM_OK ? p.bytes : 0;
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
    float *part = reinterpret_cast<float *>(ws + 2 * p.bytes);
    if (dims->batch > 0) {
        const void *states = checkpoints ? checkpoints : workspace;
        if (!checkpoints && p.nchunk > 1)   // (a single chunk starts from the initial state)
            launch_fwd<false>(x, r, g, A, nullptr, initial_state, seq_lens, nullptr, nullptr, workspace, dims, p, st);
        auto bwd = dims->io_dtype == SSM_IO_BF16 ? (p.V == 2 ? launch_bwd_v<uint16_t, 2> : launch_bwd_v<uint16_t, 1>)
                                                 : (p.V == 2 ? launch_bwd_v<float, 2> : launch_bwd_v<float, 1>);
        bwd(x, r, g, A, z, initial_state, seq_lens, dy, dlast_state, states, dx, dr, dg, dz, part, dinitial_state,
            ws + p.bytes, dims, p, st);
    }
    hipLaunchKernelGGL(ssm::column_sum_kernel, dim3((unsigned)((dims->dim + 63) / 64)),
                       dim3(64 * ssm::kColumnWaves), 0, st, part, dA, dims->batch * p.nchunk, dims->dim);
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
    const dim3 grid((unsigned)((n + 255) / 256));
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
