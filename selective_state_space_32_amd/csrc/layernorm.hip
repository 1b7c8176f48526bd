// The layer norm's entry points (include/ssmscan.h): validation and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "host_util.h"
#include "layernorm_kernel.h"

namespace {

using namespace ssmlib;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxNormDim = int64_t(1) << 30;
constexpr int64_t kMaxElems = int64_t(1) << 46;
constexpr int64_t kParts = 256;   // row blocks of the parameters' gradients

// batch * seqlen rows of dim values; dstate and chunk_len do not apply.
int check_norm_dims(const ssm_dims *dm) {
    if (!dm) return fail(SSM_ERR_NULL, "dims is NULL");
    if (dm->batch < 0 || dm->seqlen < 0 || dm->dim < 0)
        return fail(SSM_ERR_SHAPE, "negative size (batch=%lld seqlen=%lld dim=%lld)", (long long)dm->batch,
                    (long long)dm->seqlen, (long long)dm->dim);
    if (dm->io_dtype != SSM_IO_F32 && dm->io_dtype != SSM_IO_BF16)
        return fail(SSM_ERR_DTYPE, "io_dtype %d is not SSM_IO_F32 (0) or SSM_IO_BF16 (1)", dm->io_dtype);
    if (dm->batch > kMaxRows || dm->seqlen > kMaxRows || (dm->batch > 0 && dm->seqlen > kMaxRows / dm->batch))
        return fail(SSM_ERR_SHAPE, "more than 2^31 - 1 rows");
    const int64_t rows = dm->batch * dm->seqlen;
    if (dm->dim > kMaxNormDim || (rows > 0 && dm->dim > kMaxElems / rows))
        return fail(SSM_ERR_SHAPE, "dim exceeds 2^30 or the rows exceed 2^46 elements");
    return SSM_OK;
}

int check_flags(int flags) {
    if (flags & ~SSM_NORM_SUM_F32) return fail(SSM_ERR_FLAGS, "unknown flag bits 0x%x", flags);
    return SSM_OK;
}

int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    return ok();
}

int64_t part_rows(int64_t rows) { return std::max<int64_t>((rows + kParts - 1) / kParts, 1); }

template <typename IO, typename S>
void launch_norm(const void *x, const void *res, const float *w, const float *bias, float eps, void *y, void *sum,
                 float *mean, float *rstd, int64_t rows, int64_t D, hipStream_t st) {
    hipLaunchKernelGGL((ssm::layernorm_fwd_kernel<IO, S>), dim3((unsigned)rows), dim3(ssm::kNormThreads), 0, st,
                       static_cast<const IO *>(x), static_cast<const S *>(res), w, bias, eps, static_cast<IO *>(y),
                       static_cast<S *>(sum), mean, rstd, D);
}

template <typename IO, typename S>
void launch_norm_bwd(const void *dy, const void *s, const float *w, const float *mean, const float *rstd,
                     const void *dres, void *ds, void *dx, float *dw, float *db, float *part, int64_t rows, int64_t D,
                     hipStream_t st) {
    if (rows > 0)
        hipLaunchKernelGGL((ssm::layernorm_bwd_kernel<IO, S>), dim3((unsigned)rows), dim3(ssm::kNormThreads), 0, st,
                           static_cast<const IO *>(dy), static_cast<const S *>(s), w, mean, rstd,
                           static_cast<const S *>(dres), static_cast<S *>(ds), static_cast<IO *>(dx), D);
    if (!dw && !db) return;
    const int64_t per = part_rows(rows), n = (rows + per - 1) / per;
    const unsigned cols = (unsigned)((D + 255) / 256);
    if (n > 0)
        hipLaunchKernelGGL((ssm::layernorm_wgrad_kernel<IO, S>), dim3(cols, (unsigned)n), dim3(256), 0, st,
                           static_cast<const IO *>(dy), static_cast<const S *>(s), mean, rstd, part, part + n * D,
                           rows, D, per);
    hipLaunchKernelGGL(ssm::layernorm_wgrad_sum_kernel, dim3(cols), dim3(256), 0, st, part, part + n * D, dw, db, n,
                       D);
}

}  // namespace

extern "C" {

int ssm_layernorm_fwd(const void *x, const void *residual, const float *weight, const float *bias, float eps,
                      int flags, void *y, void *sum, float *mean, float *rstd, const ssm_dims *dims, void *stream) {
    int rc = check_norm_dims(dims);
    if (rc == SSM_OK) rc = check_flags(flags);
    if (rc != SSM_OK) return rc;
    if (!(eps >= 0.0f) || std::isinf(eps)) return fail(SSM_ERR_VALUE, "eps %g is negative or not finite", (double)eps);
    const size_t es = dims->io_dtype == SSM_IO_BF16 ? 2 : 4, ss = (flags & SSM_NORM_SUM_F32) ? 4 : es;
    if (!aligned(x, es) || !aligned(y, es) || !aligned(residual, ss) || !aligned(sum, ss) || !aligned(weight, 4) ||
        !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
        return fail(SSM_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    const int64_t rows = dims->batch * dims->seqlen, D = dims->dim;
    if (rows == 0 || D == 0) return ok();
    if (!x || !weight || !y) return fail(SSM_ERR_NULL, "x, weight or y is NULL");
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (es == 4)
        launch_norm<float, float>(x, residual, weight, bias, eps, y, sum, mean, rstd, rows, D, st);
    else if (ss == 4)
        launch_norm<uint16_t, float>(x, residual, weight, bias, eps, y, sum, mean, rstd, rows, D, st);
    else
        launch_norm<uint16_t, uint16_t>(x, residual, weight, bias, eps, y, sum, mean, rstd, rows, D, st);
    return launched();
}

size_t ssm_layernorm_bwd_workspace_bytes(const ssm_dims *dims) {
    if (check_norm_dims(dims) != SSM_OK) return 0;
    const int64_t rows = dims->batch * dims->seqlen, per = part_rows(rows), n = (rows + per - 1) / per;
    return align256((size_t)(2 * n * dims->dim) * sizeof(float));
}

int ssm_layernorm_bwd(const void *dy, const void *s, const float *weight, const float *mean, const float *rstd,
                      const void *dresidual, int flags, void *ds, void *dx, float *dweight, float *dbias,
                      const ssm_dims *dims, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_norm_dims(dims);
    if (rc == SSM_OK) rc = check_flags(flags);
    if (rc != SSM_OK) return rc;
    const size_t es = dims->io_dtype == SSM_IO_BF16 ? 2 : 4, ss = (flags & SSM_NORM_SUM_F32) ? 4 : es;
    if (!aligned(dy, es) || !aligned(dx, es) || !aligned(s, ss) || !aligned(dresidual, ss) || !aligned(ds, ss) ||
        !aligned(weight, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return fail(SSM_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    const int64_t rows = dims->batch * dims->seqlen, D = dims->dim;
    if (D == 0) return ok();
    if (rows > 0 && (!dy || !s || !weight || !mean || !rstd || !ds))
        return fail(SSM_ERR_NULL, "required pointer is NULL");
    const size_t need = dweight || dbias ? ssm_layernorm_bwd_workspace_bytes(dims) : 0;
    if (need > 0 && !workspace) return fail(SSM_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (workspace_bytes < need)
        return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes, need);
    if (need > 0 && !aligned(workspace, 16)) return fail(SSM_ERR_ALIGN, "workspace not 16-byte aligned");
    hipStream_t st = static_cast<hipStream_t>(stream);
    float *part = static_cast<float *>(workspace);
    if (es == 4)
        launch_norm_bwd<float, float>(dy, s, weight, mean, rstd, dresidual, ds, dx, dweight, dbias, part, rows, D, st);
    else if (ss == 4)
        launch_norm_bwd<uint16_t, float>(dy, s, weight, mean, rstd, dresidual, ds, dx, dweight, dbias, part, rows, D,
                                         st);
    else
        launch_norm_bwd<uint16_t, uint16_t>(dy, s, weight, mean, rstd, dresidual, ds, dx, dweight, dbias, part, rows,
                                            D, st);
    return launched();
}

}  // extern "C"
