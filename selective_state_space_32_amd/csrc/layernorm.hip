// The layer norm's entry points (include/ssmscan.h): validation and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "host_util.h"
#include "layernorm_kernel.h"

namespace {

using namespace ssmlib;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxNormDim = int64_t(1) << 26;   // (the column sums launch 32 threads per column)
constexpr int64_t kMaxElems = int64_t(1) << 46;
constexpr int64_t kWideGroups = int64_t(1) << 16;   // workgroups of the kernels for wider rows, at most
constexpr int64_t kWideParts = 256;   // partial sums for rows wider than the registers hold

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
        return fail(SSM_ERR_SHAPE, "dim exceeds 2^26 or the rows exceed 2^46 elements");
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

// Workgroups of the forward, at most.  A workgroup takes several rows, so that its weights are worth
// keeping: two per CU for wide rows (16384x5120 bf16 with an fp32 residual: 177 us, 185 with four), four
// for narrow ones, of which a workgroup requests fewer bytes at a time (32768x500: 40 us, 60 with two).
int64_t fwd_groups(int64_t D) { return D <= 2048 ? 1024 : 512; }

// The widest rows that the forward holds in registers (of 1024 threads: 4096x12288 bf16 with fp32 sums, 106
// us; passing over the row three times takes 142).
constexpr int64_t kFwdDim = 16384;

// Rows that a workgroup holds at a time (a wave each, up to 1024 values), by the row's width (0: wider
// than the backward's registers hold).
int64_t norm_slots(int64_t D) { return D <= 1024 ? 4 : D <= 8192 ? 1 : 0; }

// Rows start on 128-byte lines (of tensors that do).
bool whole_lines(int64_t D, int64_t es) { return D * es % 128 == 0; }

// Workgroups of the backward, at most, and so partial sums of the parameters' gradients.  Two per CU
// (16384x5120 bf16, fp32 sums: 225 us and 5 for the sums with 512; 264 + 5 with 256, 237 + 8 with 1024;
// 32768x768: 71 + 5 and 74 + 6; a wave per SIMD is all that the registers of 2049 to 5120 fp32 values admit,
// half of 512 workgroups at a time: 16384x5120 fp32, fp32 sums 257 + 5), four for the narrowest rows, which
// request few bytes at a time (32768x200: 30 + 5 us with 512, 21 + 6 with 1024), and for narrow ones that go
// through the caches (32768x1500: 213 + 5 and 152 + 7; whole lines, 16384x2048: 88 + 5 and 98 + 6).
int64_t bwd_groups(int64_t D, int64_t es) {
    return D <= 256 || (D > 1024 && D <= 2048 && !whole_lines(D, es)) ? 1024 : 512;
}
int64_t norm_parts(int64_t rows, int64_t D, int64_t es) {
    const int64_t slots = norm_slots(D);
    if (slots == 0) return std::min<int64_t>(rows, kWideParts);
    return std::min<int64_t>((rows + slots - 1) / slots, bwd_groups(D, es));
}

// The narrowest shape that holds a row of D values: lanes past the row's end do nothing.
template <typename IO, typename S, bool NT>
auto fwd_kernel_of(int64_t D) {
    return D <= 256    ? ssm::layernorm_fwd_kernel<IO, S, 64, 1, NT>
           : D <= 1024 ? ssm::layernorm_fwd_kernel<IO, S, 64, 4, NT>
           : D <= 2048 ? ssm::layernorm_fwd_kernel<IO, S, 256, 2, NT>
           : D <= 5120 ? ssm::layernorm_fwd_kernel<IO, S, 256, 5, NT>
           : D <= 8192 ? ssm::layernorm_fwd_kernel<IO, S, 256, 8, NT>
                       : ssm::layernorm_fwd_kernel<IO, S, 1024, 4, NT>;
}
template <typename IO, typename S, bool NT>
auto bwd_kernel_of(int64_t D) {
    return D <= 256    ? ssm::layernorm_bwd_kernel<IO, S, 64, 1, NT>
           : D <= 1024 ? ssm::layernorm_bwd_kernel<IO, S, 64, 4, NT>
           : D <= 2048 ? ssm::layernorm_bwd_kernel<IO, S, 256, 2, NT>
           : D <= 5120 ? ssm::layernorm_bwd_kernel<IO, S, 256, 5, NT>
                       : ssm::layernorm_bwd_kernel<IO, S, 512, 4, NT>;
}

template <typename IO, typename S>
void launch_norm(const void *x_, const void *res_, const float *w, const float *bias, float eps, void *y_, void *sum_,
                 float *mean, float *rstd, int64_t rows, int64_t D, hipStream_t st) {
    const IO *x = static_cast<const IO *>(x_);
    const S *res = static_cast<const S *>(res_);
    IO *y = static_cast<IO *>(y_);
    S *sum = static_cast<S *>(sum_);
    if (D > kFwdDim) {
        hipLaunchKernelGGL((ssm::layernorm_fwd_wide_kernel<IO, S>), dim3((unsigned)std::min(rows, kWideGroups)),
                           dim3(ssm::kNormWideThreads), 0, st, x, res, w, bias, eps, y, sum, mean, rstd, rows, D);
        return;
    }
    auto kern = whole_lines(D, sizeof(IO)) ? fwd_kernel_of<IO, S, true>(D) : fwd_kernel_of<IO, S, false>(D);
    const int64_t slots = std::max<int64_t>(norm_slots(D), 1);
    const int64_t grid = std::min<int64_t>((rows + slots - 1) / slots, fwd_groups(D));
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(D <= 8192 ? 256 : 1024), 0, st, x, res, w, bias, eps, y, sum,
                       mean, rstd, rows, D);
}

template <typename IO, typename S>
void launch_norm_bwd(const void *dy_, const void *s_, const float *w, const float *mean, const float *rstd,
                     const void *dres_, void *ds_, void *dx_, float *dw, float *db, float *part, int64_t rows,
                     int64_t D, hipStream_t st) {
    const IO *dy = static_cast<const IO *>(dy_);
    const S *s = static_cast<const S *>(s_), *dres = static_cast<const S *>(dres_);
    S *ds = static_cast<S *>(ds_);
    IO *dx = static_cast<IO *>(dx_);
    const int64_t parts = norm_parts(rows, D, sizeof(IO));
    const bool sums = dw || db;   // (without rows there are no parts: the sums are zero)
    float *pw = sums ? part : nullptr, *pb = sums ? part + parts * D : nullptr;
    if (rows > 0 && norm_slots(D) == 0) {
        hipLaunchKernelGGL((ssm::layernorm_bwd_wide_kernel<IO, S>), dim3((unsigned)std::min(rows, kWideGroups)),
                           dim3(ssm::kNormWideThreads), 0, st, dy, s, w, mean, rstd, dres, ds, dx, rows, D);
    } else if (rows > 0) {
        auto kern = whole_lines(D, sizeof(IO)) ? bwd_kernel_of<IO, S, true>(D) : bwd_kernel_of<IO, S, false>(D);
        hipLaunchKernelGGL(kern, dim3((unsigned)parts), dim3(D <= 5120 ? 256 : 512), 0, st, dy, s, w, mean, rstd,
                           dres, ds, dx, pw, pb, rows, D);
    }
    if (!sums) return;
    if (rows > 0 && norm_slots(D) == 0) {
        // ds may have replaced dresidual, but dy and s are still there
        const int64_t per = (rows + parts - 1) / parts;
        hipLaunchKernelGGL((ssm::layernorm_wgrad_wide_kernel<IO, S>),
                           dim3((unsigned)((D + 256 * ssm::kNormVec - 1) / (256 * ssm::kNormVec)), (unsigned)parts),
                           dim3(256), 0, st, dy, s, mean, rstd, pw, pb, rows, D, per);
    }
    hipLaunchKernelGGL(ssm::layernorm_wgrad_sum_kernel,
                       dim3((unsigned)((D + ssm::kNormSumCols - 1) / ssm::kNormSumCols)),
                       dim3(ssm::kNormSumCols * ssm::kNormSumGroups), 0, st, pw, pb, dw, db, parts, D);
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
    // (rows without values still have statistics: a mean of 0 / 0)
    if (rows == 0 || (D == 0 && !mean && !rstd)) return ok();
    if (D > 0 && (!x || !weight || !y)) return fail(SSM_ERR_NULL, "x, weight or y is NULL");
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
    const int64_t es = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
    return align256((size_t)(2 * norm_parts(dims->batch * dims->seqlen, dims->dim, es) * dims->dim) * sizeof(float));
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
