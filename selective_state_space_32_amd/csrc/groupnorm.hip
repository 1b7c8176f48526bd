// The group norm's entry points (include/ssmscan.h): validation and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "groupnorm_kernel.h"
#include "host_util.h"

namespace {

using namespace ssmlib;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxNormDim = int64_t(1) << 26;   // (the column sums launch 32 threads per column)
constexpr int64_t kMaxElems = int64_t(1) << 46;
constexpr int64_t kRegDim = 8192;                   // the widest groups that are held in registers
constexpr int64_t kWideGroups = int64_t(1) << 16;   // workgroups of the kernels for wider ones, at most
constexpr int64_t kWideParts = 256;                 // and their partial sums of the parameters' gradients
constexpr int kFlags = SSM_GROUPNORM_RMS | SSM_GROUPNORM_GATE_FIRST | SSM_GROUPNORM_SILU;

int check_dims(const ssm_dims *dm, int64_t groups, int flags, const void *z, int64_t z_stride) {
    if (!dm) return fail(SSM_ERR_NULL, "dims is NULL");
    if (dm->batch < 0 || dm->seqlen < 0 || dm->dim < 0)
        return fail(SSM_ERR_SHAPE, "negative size (batch=%lld seqlen=%lld dim=%lld)", (long long)dm->batch,
                    (long long)dm->seqlen, (long long)dm->dim);
    if (dm->io_dtype != SSM_IO_F32 && dm->io_dtype != SSM_IO_BF16)
        return fail(SSM_ERR_DTYPE, "io_dtype %d is not SSM_IO_F32 (0) or SSM_IO_BF16 (1)", dm->io_dtype);
    if (groups < 1 || dm->dim % groups)
        return fail(SSM_ERR_SHAPE, "dim %lld is not a multiple of groups %lld", (long long)dm->dim, (long long)groups);
    if (dm->batch > kMaxRows || dm->seqlen > kMaxRows || (dm->batch > 0 && dm->seqlen > kMaxRows / dm->batch))
        return fail(SSM_ERR_SHAPE, "more than 2^31 - 1 rows");
    const int64_t rows = dm->batch * dm->seqlen;
    if (dm->dim > kMaxNormDim || z_stride > (int64_t(1) << 30) || (rows > 0 && std::max(dm->dim, z_stride) > kMaxElems / rows))
        return fail(SSM_ERR_SHAPE, "dim exceeds 2^26, z_stride 2^30, or the rows 2^46 elements");
    if (flags & ~kFlags) return fail(SSM_ERR_FLAGS, "unknown flag bits 0x%x", flags);
    if ((flags & SSM_GROUPNORM_GATE_FIRST) && !z) return fail(SSM_ERR_NULL, "SSM_GROUPNORM_GATE_FIRST without z");
    if ((flags & SSM_GROUPNORM_SILU) && z) return fail(SSM_ERR_FLAGS, "SSM_GROUPNORM_SILU together with z");
    if (z && z_stride != 0 && z_stride < dm->dim)
        return fail(SSM_ERR_SHAPE, "z_stride %lld is smaller than dim %lld", (long long)z_stride, (long long)dm->dim);
    return SSM_OK;
}

int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    return ok();
}

// Threads per group (and vectors of four values per thread) by the group's width: the fewest that hold it.
int group_threads(int64_t D) { return D <= 32 ? 8 : D <= 64 ? 16 : D <= 128 ? 32 : D <= 1024 ? 64 : D <= 5120 ? 256 : 512; }

// Workgroups, at most: they take several rows each, so that the weights they hold are worth it; as many as the chip
// holds at once, or nearly (16384x5120 bf16, 8 groups, gate first: forward 115 us with 1024, 102 with 1536, 111 with
// 4096; backward 286 with 512, 218 with 768, 192 with 1024, which fit where a thread holds up to three vectors).
constexpr int64_t kFwdGroups = 1536;
int64_t bwd_groups(int64_t D) { return D <= 768 || (D > 1024 && D <= 2048) ? 1024 : 512; }

// (of rows with values: their groups are at most dim, which an int holds)
ssm::gn_shape shape_of(const ssm_dims *dm, int64_t groups, int64_t z_stride, int flags, const void *z) {
    ssm::gn_shape s;
    s.M = dm->batch * dm->seqlen;
    s.C = dm->dim;
    s.D = dm->dim / groups;
    s.zs = z_stride ? z_stride : dm->dim;
    s.G = (int)groups;
    const int tpg = group_threads(s.D), slots = tpg >= 256 ? 1 : 256 / tpg;
    s.gblocks = (s.G + slots - 1) / slots;
    s.spr = (s.G + s.gblocks - 1) / s.gblocks;
    s.rpb = std::max(slots / s.spr, 1);
    s.act = flags & SSM_GROUPNORM_SILU ? ssm::kGnSilu : !z ? ssm::kGnPlain : flags & SSM_GROUPNORM_GATE_FIRST ? ssm::kGnGateFirst : ssm::kGnGateAfter;
    s.centre = flags & SSM_GROUPNORM_RMS ? 0 : 1;
    return s;
}

// Workgroups along the rows; parts of the parameters' sums: one per row that a workgroup takes at a time.
int64_t row_blocks(const ssm::gn_shape &s, int64_t most) {
    return std::max<int64_t>(std::min<int64_t>((s.M + s.rpb - 1) / s.rpb, most / s.gblocks), 1);
}
int64_t norm_parts(const ssm::gn_shape &s) {
    if (s.M == 0) return 0;
    return s.D > kRegDim ? std::min<int64_t>(s.M, kWideParts) : row_blocks(s, bwd_groups(s.D)) * s.rpb;
}

template <typename IO, int ACT> auto fwd_kernel_of(int64_t D) {
    return D <= 32   ? ssm::groupnorm_fwd_kernel<IO, 8, 1, ACT>
         : D <= 64   ? ssm::groupnorm_fwd_kernel<IO, 16, 1, ACT>
         : D <= 128  ? ssm::groupnorm_fwd_kernel<IO, 32, 1, ACT>
         : D <= 256  ? ssm::groupnorm_fwd_kernel<IO, 64, 1, ACT>
         : D <= 512  ? ssm::groupnorm_fwd_kernel<IO, 64, 2, ACT>
         : D <= 768  ? ssm::groupnorm_fwd_kernel<IO, 64, 3, ACT>
         : D <= 1024 ? ssm::groupnorm_fwd_kernel<IO, 64, 4, ACT>
         : D <= 2048 ? ssm::groupnorm_fwd_kernel<IO, 256, 2, ACT>
         : D <= 5120 ? ssm::groupnorm_fwd_kernel<IO, 256, 5, ACT>
                      : ssm::groupnorm_fwd_kernel<IO, 512, 4, ACT>;
}
template <typename IO, int ACT> auto bwd_kernel_of(int64_t D) {
    return D <= 32   ? ssm::groupnorm_bwd_kernel<IO, 8, 1, ACT>
         : D <= 64   ? ssm::groupnorm_bwd_kernel<IO, 16, 1, ACT>
         : D <= 128  ? ssm::groupnorm_bwd_kernel<IO, 32, 1, ACT>
         : D <= 256  ? ssm::groupnorm_bwd_kernel<IO, 64, 1, ACT>
         : D <= 512  ? ssm::groupnorm_bwd_kernel<IO, 64, 2, ACT>
         : D <= 768  ? ssm::groupnorm_bwd_kernel<IO, 64, 3, ACT>
         : D <= 1024 ? ssm::groupnorm_bwd_kernel<IO, 64, 4, ACT>
         : D <= 2048 ? ssm::groupnorm_bwd_kernel<IO, 256, 2, ACT>
         : D <= 5120 ? ssm::groupnorm_bwd_kernel<IO, 256, 5, ACT>
                      : ssm::groupnorm_bwd_kernel<IO, 512, 4, ACT>;
}
template <typename IO> auto fwd_kernel_of(const ssm::gn_shape &s) {
    return s.act == ssm::kGnPlain       ? fwd_kernel_of<IO, ssm::kGnPlain>(s.D)
         : s.act == ssm::kGnGateFirst ? fwd_kernel_of<IO, ssm::kGnGateFirst>(s.D)
         : s.act == ssm::kGnGateAfter ? fwd_kernel_of<IO, ssm::kGnGateAfter>(s.D)
                                      : fwd_kernel_of<IO, ssm::kGnSilu>(s.D);
}
template <typename IO> auto bwd_kernel_of(const ssm::gn_shape &s) {
    return s.act == ssm::kGnPlain       ? bwd_kernel_of<IO, ssm::kGnPlain>(s.D)
         : s.act == ssm::kGnGateFirst ? bwd_kernel_of<IO, ssm::kGnGateFirst>(s.D)
         : s.act == ssm::kGnGateAfter ? bwd_kernel_of<IO, ssm::kGnGateAfter>(s.D)
                                      : bwd_kernel_of<IO, ssm::kGnSilu>(s.D);
}

template <typename IO>
void launch_fwd(const void *x_, const void *z_, const float *w, const float *bias, float eps, void *y_, float *mean,
                float *rstd, const ssm::gn_shape &s, hipStream_t st) {
    const IO *x = static_cast<const IO *>(x_), *z = static_cast<const IO *>(z_);
    IO *y = static_cast<IO *>(y_);
    if (s.D > kRegDim) {
        hipLaunchKernelGGL(ssm::groupnorm_fwd_wide_kernel<IO>, dim3((unsigned)std::min(s.M * s.G, kWideGroups)),
                           dim3(ssm::kNormWideThreads), 0, st, x, z, w, bias, eps, y, mean, rstd, s);
        return;
    }
    hipLaunchKernelGGL(fwd_kernel_of<IO>(s), dim3((unsigned)(row_blocks(s, kFwdGroups) * s.gblocks)),
                       dim3(std::max(group_threads(s.D), 256)), 0, st, x, z, w, bias, eps, y, mean, rstd, s);
}

template <typename IO>
void launch_bwd(const void *dy_, const void *x_, const void *z_, const float *w, const float *bias, const float *mean,
                const float *rstd, void *dx_, void *dz_, float *dw, float *db, float *part, const ssm::gn_shape &s,
                hipStream_t st) {
    const IO *dy = static_cast<const IO *>(dy_), *x = static_cast<const IO *>(x_), *z = static_cast<const IO *>(z_);
    IO *dx = static_cast<IO *>(dx_), *dz = static_cast<IO *>(dz_);
    const int64_t parts = norm_parts(s);
    const bool sums = dw || db;   // (without rows there are no parts: the sums are zero)
    float *pw = sums ? part : nullptr, *pb = sums ? part + parts * s.C : nullptr;
    if (s.M > 0 && s.D > kRegDim) {
        hipLaunchKernelGGL(ssm::groupnorm_bwd_wide_kernel<IO>, dim3((unsigned)std::min(s.M * s.G, kWideGroups)),
                           dim3(ssm::kNormWideThreads), 0, st, dy, x, z, w, bias, mean, rstd, dx, dz, s);
        if (sums) {
            const int64_t per = (s.M + parts - 1) / parts, vecs = (s.D + ssm::kNormVec - 1) / ssm::kNormVec * s.G;
            hipLaunchKernelGGL(ssm::groupnorm_wgrad_wide_kernel<IO>, dim3((unsigned)((vecs + 255) / 256), (unsigned)parts),
                               dim3(256), 0, st, dy, x, z, w, bias, mean, rstd, pw, pb, s, per);
        }
    } else if (s.M > 0) {
        hipLaunchKernelGGL(bwd_kernel_of<IO>(s), dim3((unsigned)(row_blocks(s, bwd_groups(s.D)) * s.gblocks)),
                           dim3(std::max(group_threads(s.D), 256)), 0, st, dy, x, z, w, bias, mean, rstd, dx, dz, pw, pb, s);
    }
    if (sums)
        hipLaunchKernelGGL(ssm::layernorm_wgrad_sum_kernel, dim3((unsigned)((s.C + ssm::kNormSumCols - 1) / ssm::kNormSumCols)),
                           dim3(ssm::kNormSumCols * ssm::kNormSumGroups), 0, st, pw, pb, dw, db, parts, s.C);
}

}  // namespace

extern "C" {

int ssm_groupnorm_fwd(const void *x, const void *z, int64_t z_stride, const float *weight, const float *bias, int64_t groups,
                      float eps, int flags, void *y, float *mean, float *rstd, const ssm_dims *dims, void *stream) {
    const int rc = check_dims(dims, groups, flags, z, z_stride);
    if (rc != SSM_OK) return rc;
    if (!(eps >= 0.0f) || std::isinf(eps)) return fail(SSM_ERR_VALUE, "eps %g is negative or not finite", (double)eps);
    const size_t es = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
    if (!aligned(x, es) || !aligned(z, es) || !aligned(y, es) || !aligned(weight, 4) || !aligned(bias, 4) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return fail(SSM_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    if (dims->batch == 0 || dims->seqlen == 0 || dims->dim == 0) return ok();   // (nothing is of any number of groups)
    const ssm::gn_shape s = shape_of(dims, groups, z_stride, flags, z);
    if (!x || !weight || !y) return fail(SSM_ERR_NULL, "x, weight or y is NULL");
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (es == 2) launch_fwd<uint16_t>(x, z, weight, bias, eps, y, mean, rstd, s, st);
    else launch_fwd<float>(x, z, weight, bias, eps, y, mean, rstd, s, st);
    return launched();
}

size_t ssm_groupnorm_bwd_workspace_bytes(const ssm_dims *dims, int64_t groups) {
    if (check_dims(dims, groups, 0, nullptr, 0) != SSM_OK || dims->dim == 0) return 0;
    return align256((size_t)(2 * norm_parts(shape_of(dims, groups, 0, 0, nullptr)) * dims->dim) * sizeof(float));
}

int ssm_groupnorm_bwd(const void *dy, const void *x, const void *z, int64_t z_stride, const float *weight, const float *bias,
                      const float *mean, const float *rstd, int64_t groups, int flags, void *dx, void *dz, float *dweight,
                      float *dbias, const ssm_dims *dims, void *workspace, size_t workspace_bytes, void *stream) {
    const int rc = check_dims(dims, groups, flags, z, z_stride);
    if (rc != SSM_OK) return rc;
    const size_t es = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
    if (!aligned(dy, es) || !aligned(x, es) || !aligned(z, es) || !aligned(dx, es) || !aligned(dz, es) || !aligned(weight, 4) ||
        !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return fail(SSM_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    if (dims->dim == 0) return ok();
    const ssm::gn_shape s = shape_of(dims, groups, z_stride, flags, z);
    if (s.M > 0 && (!dy || !x || !weight || !rstd || !dx || (s.centre && !mean) || (z && !dz)))
        return fail(SSM_ERR_NULL, "required pointer is NULL");
    const size_t need = dweight || dbias ? ssm_groupnorm_bwd_workspace_bytes(dims, groups) : 0;
    if (need > 0 && !workspace) return fail(SSM_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (workspace_bytes < need)
        return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes, need);
    if (need > 0 && !aligned(workspace, 16)) return fail(SSM_ERR_ALIGN, "workspace not 16-byte aligned");
    hipStream_t st = static_cast<hipStream_t>(stream);
    float *part = static_cast<float *>(workspace);
    if (es == 2) launch_bwd<uint16_t>(dy, x, z, weight, bias, mean, rstd, dx, dz, dweight, dbias, part, s, st);
    else launch_bwd<float>(dy, x, z, weight, bias, mean, rstd, dx, dz, dweight, dbias, part, s, st);
    return launched();
}

}  // extern "C"
