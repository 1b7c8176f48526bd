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

size_t states_bytes(const ssm_dims *dm) {
    const int64_t n = (dm->seqlen + ssm::kGatedCkpt - 1) / ssm::kGatedCkpt;
    return align256((size_t)(dm->batch * n * dm->dim) * sizeof(float));
}

template <typename IO>
void launch_fwd(const void *x, const void *r, const void *g, const float *A, const void *z, const float *h0,
                const int32_t *sl, void *y, float *last, float *ckpt, const ssm_dims *dm, hipStream_t st) {
    const int64_t tiles = (dm->dim + 63) / 64;
    hipLaunchKernelGGL(ssm::gated_scan_kernel<IO>, dim3((unsigned)(dm->batch * tiles)), dim3(64), 0, st,
                       static_cast<const IO *>(x), static_cast<const IO *>(r), static_cast<const IO *>(g), A,
                       static_cast<const IO *>(z), h0, sl, static_cast<IO *>(y), last, ckpt, dm->seqlen, dm->dim,
                       tiles);
}

template <typename IO>
void launch_bwd(const void *x, const void *r, const void *g, const float *A, const void *z, const int32_t *sl,
                const void *dy, const float *dlast, const float *ckpt, void *dx, void *dr, void *dg, float *dA,
                void *dz, float *dh0, float *part, const ssm_dims *dm, hipStream_t st) {
    const int64_t tiles = (dm->dim + 63) / 64;
    if (dm->batch > 0)
        hipLaunchKernelGGL(ssm::gated_bwd_kernel<IO>, dim3((unsigned)(dm->batch * tiles)), dim3(64), 0, st,
                           static_cast<const IO *>(x), static_cast<const IO *>(r), static_cast<const IO *>(g), A,
                           static_cast<const IO *>(z), sl, static_cast<const IO *>(dy), dlast, ckpt,
                           static_cast<IO *>(dx), static_cast<IO *>(dr), static_cast<IO *>(dg), static_cast<IO *>(dz),
                           part, dh0, dm->seqlen, dm->dim, tiles);
    hipLaunchKernelGGL(ssm::column_sum_kernel, dim3((unsigned)((dm->dim + 255) / 256)), dim3(256), 0, st, part, dA,
                       dm->batch, dm->dim);
}

}  // namespace

extern "C" {

size_t ssm_gated_scan_workspace_bytes(const ssm_dims *dims) {
    if (check_gated_dims(dims, true) != SSM_OK) return 0;
    return states_bytes(dims);
}

size_t ssm_gated_scan_bwd_workspace_bytes(const ssm_dims *dims) {
    if (check_gated_dims(dims, true) != SSM_OK) return 0;
    return states_bytes(dims) + align256((size_t)(dims->batch * dims->dim) * sizeof(float));
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
    const size_t need = states_bytes(dims);
    if (need > 0 && !workspace) return fail(SSM_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (workspace_bytes < need)
        return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes, need);
    if (need > 0 && !aligned(workspace, 16)) return fail(SSM_ERR_ALIGN, "workspace not 16-byte aligned");
    hipStream_t st = static_cast<hipStream_t>(stream);
    float *ckpt = static_cast<float *>(workspace);
    if (es == 2)
        launch_fwd<uint16_t>(x, r, g, A, z, initial_state, seq_lens, y, last_state, ckpt, dims, st);
    else
        launch_fwd<float>(x, r, g, A, z, initial_state, seq_lens, y, last_state, ckpt, dims, st);
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
    if (dims->batch > 0) {
        if (!A || (dims->seqlen > 0 && (!x || !r || !g || !dy || !dx || !dr || !dg)))
            return fail(SSM_ERR_NULL, "required pointer is NULL");
        if (dims->seqlen > 0 && z && !dz) return fail(SSM_ERR_NULL, "z is given but dz is NULL");
        const size_t need = ssm_gated_scan_bwd_workspace_bytes(dims), ck = states_bytes(dims);
        if (need > 0 && !workspace) return fail(SSM_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
        if (workspace_bytes < need)
            return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes,
                        need);
        if (checkpoints && checkpoints_bytes < ck)
            return fail(SSM_ERR_WORKSPACE, "checkpoints of %zu bytes are smaller than the %zu needed",
                        checkpoints_bytes, ck);
        if (!aligned(workspace, 16) || !aligned(checkpoints, 16))
            return fail(SSM_ERR_ALIGN, "workspace or checkpoints not 16-byte aligned");
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    float *part = reinterpret_cast<float *>(static_cast<char *>(workspace) + states_bytes(dims));
    const float *ckpt = static_cast<const float *>(checkpoints ? checkpoints : workspace);
    if (dims->batch > 0 && !checkpoints) {
        if (es == 2)
            launch_fwd<uint16_t>(x, r, g, A, nullptr, initial_state, seq_lens, nullptr, nullptr,
                                 static_cast<float *>(workspace), dims, st);
        else
            launch_fwd<float>(x, r, g, A, nullptr, initial_state, seq_lens, nullptr, nullptr,
                              static_cast<float *>(workspace), dims, st);
    }
    if (es == 2)
        launch_bwd<uint16_t>(x, r, g, A, z, seq_lens, dy, dlast_state, ckpt, dx, dr, dg, dA, dz, dinitial_state, part,
                             dims, st);
    else
        launch_bwd<float>(x, r, g, A, z, seq_lens, dy, dlast_state, ckpt, dx, dr, dg, dA, dz, dinitial_state, part,
                          dims, st);
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
