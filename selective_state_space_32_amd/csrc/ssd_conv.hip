// The state space dual layer with its convolution (include/ssmscan.h): validation and launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "host_util.h"
#include "ssd_conv_bwd_kernel.h"
#include "ssd_conv_kernel.h"

namespace {

using namespace ssmlib;

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxElems = int64_t(1) << 46;
// Workgroups of a launch at most: HIP refuses 2^32 threads or more in a dimension.
constexpr int64_t max_groups(int threads) { return ((int64_t(1) << 32) - 1) / threads; }

int64_t row_of(const ssm_ssd_conv_dims *dm) { return dm->nheads * dm->headdim + 2 * dm->ngroups * dm->dstate; }
size_t elem_size(const ssm_ssd_conv_dims *dm) { return dm->io_dtype == SSM_IO_BF16 ? 2 : 4; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t p_tiles(const ssm_ssd_conv_dims *dm) { return ceil_div(dm->headdim, 64); }
int64_t chunks(const ssm_ssd_conv_dims *dm) { return ceil_div(dm->seqlen, ssm::kSdQ); }

int check_dims(const ssm_ssd_conv_dims *dm) {
    if (!dm) return fail(SSM_ERR_NULL, "dims is NULL");
    if (dm->batch < 0 || dm->seqlen < 0 || dm->nheads < 0)
        return fail(SSM_ERR_SHAPE, "negative size (batch=%lld seqlen=%lld nheads=%lld)", (long long)dm->batch,
                    (long long)dm->seqlen, (long long)dm->nheads);
    if (dm->io_dtype != SSM_IO_F32 && dm->io_dtype != SSM_IO_BF16)
        return fail(SSM_ERR_DTYPE, "io_dtype %d is not SSM_IO_F32 (0) or SSM_IO_BF16 (1)", dm->io_dtype);
    if (dm->headdim < 8 || dm->headdim % 8 || dm->headdim > 65536)
        return fail(SSM_ERR_SHAPE, "headdim %lld is not a multiple of 8 from 8 to 65536", (long long)dm->headdim);
    if (dm->dstate < 8 || dm->dstate % 8 || dm->dstate > 128)
        return fail(SSM_ERR_SHAPE, "dstate %lld is not a multiple of 8 from 8 to 128", (long long)dm->dstate);
    if (dm->ngroups < 1 || dm->nheads % dm->ngroups)
        return fail(SSM_ERR_SHAPE, "nheads %lld is not a multiple of ngroups %lld", (long long)dm->nheads, (long long)dm->ngroups);
    if (dm->width < 1 || dm->width > ssm::kSdTaps)
        return fail(SSM_ERR_SHAPE, "convolution width %d is not 1 to %d", dm->width, ssm::kSdTaps);
    // (64 rows of u, at most 2^23 elements each, are addressed by 32-bit offsets)
    if (dm->nheads > (int64_t(1) << 22) / dm->headdim || dm->ngroups > (int64_t(1) << 21) / dm->dstate)
        return fail(SSM_ERR_SHAPE, "nheads*headdim or 2*ngroups*dstate exceeds 2^22");
    if (dm->seqlen > kMaxTokens || dm->batch > kMaxTokens)
        return fail(SSM_ERR_SHAPE, "seqlen or batch exceeds 2^30");
    const int64_t row = row_of(dm);
    if (dm->nheads > 0 && dm->batch > 0 &&
        (dm->batch > kMaxElems / row / std::max<int64_t>(dm->seqlen, 1) ||
         dm->batch > kMaxElems / (dm->nheads * dm->headdim * dm->dstate) / std::max<int64_t>(chunks(dm), 1)))
        return fail(SSM_ERR_SHAPE, "the rows or the states exceed 2^46 elements");
    if (dm->xbc_stride < 0 || dm->dt_stride < 0 || (dm->xbc_stride && dm->xbc_stride < row) ||
        (dm->dt_stride && dm->dt_stride < dm->nheads) || dm->xbc_stride > kMaxTokens || dm->dt_stride > kMaxTokens)
        return fail(SSM_ERR_SHAPE, "a stride between tokens is smaller than the row or larger than 2^30");
    return SSM_OK;
}

int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    return ok();
}

// Segments of a sequence, which run beside each other: a pass over the state alone finds what each of them starts
// from.  One, unless the sequences' heads leave most of the workgroups that fit on the chip without work; at least two
// chunks each.  (All passes, B1 L65536 H32 N128: 567 us, 4,658 as one segment; B5 L777 H20 N128: 47 and 70; B1 L512 H24
// N64: 21 and 32; B2 L2048 H24 fp32: 68 and 197.  768 to 1,536 in place of 512 are no better: 583 to 633 for the first, 65
// to 66 for the last.)
constexpr int64_t kSegTarget = 512;
int64_t segments(const ssm_ssd_conv_dims *dm) {
    const int64_t items = dm->batch * dm->nheads * p_tiles(dm), most = std::max<int64_t>(chunks(dm) / 2, 1);
    return std::min(std::max<int64_t>(kSegTarget / std::max<int64_t>(items, 1), 1), most);
}

ssm::sd_shape shape_of(const ssm_ssd_conv_dims *dm, int flags) {
    ssm::sd_shape s;
    s.L = dm->seqlen;
    s.H = (int)dm->nheads;
    s.P = (int)dm->headdim;
    s.G = (int)dm->ngroups;
    s.N = (int)dm->dstate;
    s.PT = (int)p_tiles(dm);
    s.dc = (int)row_of(dm);
    s.dt_stride = dm->dt_stride ? dm->dt_stride : dm->nheads;
    s.softplus = flags & SSM_SCAN_SOFTPLUS;
    s.nchunk = chunks(dm);
    s.cps = std::max<int64_t>(ceil_div(s.nchunk, segments(dm)), 1);
    s.nseg = (int)std::max<int64_t>(ceil_div(s.nchunk, s.cps), 1);
    return s;
}

// The workspace of the forward: u, the tokens' decays, and in training the states entering the chunks.
size_t u_bytes(const ssm_ssd_conv_dims *dm) { return align256((size_t)(dm->batch * dm->seqlen * row_of(dm)) * elem_size(dm)); }
size_t tok_bytes(const ssm_ssd_conv_dims *dm) { return align256((size_t)(dm->batch * dm->nheads * chunks(dm) * ssm::kSdTok) * sizeof(float)); }
size_t state_bytes(const ssm_ssd_conv_dims *dm) {
    return align256((size_t)(dm->batch * chunks(dm) * dm->nheads * dm->headdim * dm->dstate) * sizeof(float));
}

// The segments' states (none where there is one segment).
size_t seg_bytes(const ssm_ssd_conv_dims *dm) {
    const int64_t n = shape_of(dm, 0).nseg;
    return n > 1 ? align256((size_t)(dm->batch * dm->nheads * n * dm->headdim * dm->dstate) * sizeof(float)) : 0;
}

// Tokens per thread of the convolution: 32 (a thread reads three rows more than it has), 8 where that leaves CUs
// with less than four waves per SIMD (B8 L2048 of 5,248 channels bf16: 96 us, 127 with 8; B1 L512 of 1,664: 8.2 us with
// 8, 17.7 with 32; B5 L777 of 2,304: 20 and 28; B2 L2048 of 1,664 fp32: 16.6 and 14.8).
int conv_tokens(const ssm_ssd_conv_dims *dm) {
    return dm->batch * dm->seqlen * (row_of(dm) / ssm::kSdConvV) >= (int64_t)32 * 64 * 4096 ? 32 : 8;
}
struct ConvGrid {
    int64_t vblocks, tiles, blocks, quads;   // workgroups of the convolution: vblocks * tiles * batch; then the tokens'
    bool fits() const { return blocks + quads <= max_groups(256); }
};
ConvGrid conv_grid(const ssm_ssd_conv_dims *dm, int tt, bool tokens) {
    ConvGrid g;
    g.vblocks = ceil_div(row_of(dm) / ssm::kSdConvV, 256);
    g.tiles = std::max<int64_t>(ceil_div(dm->seqlen, tt), 1);
    g.blocks = g.vblocks * g.tiles * dm->batch;
    g.quads = tokens ? dm->batch * chunks(dm) * ceil_div(dm->nheads, 4) : 0;
    return g;
}

// Whether the forward's launches can be made (the last of them as well as the first: none is made otherwise).
int check_forward(const ssm_ssd_conv_dims *dm) {
    const int rc = check_dims(dm);
    if (rc != SSM_OK || dm->batch == 0 || dm->nheads == 0) return rc;
    if (dm->nheads * p_tiles(dm) > max_groups(ssm::kSdThreads) / dm->batch)   // (segments only add to less than kSegTarget)
        return fail(SSM_ERR_SHAPE, "batch*nheads*ceil(headdim/64) exceeds %lld, the workgroups of a launch",
                    (long long)max_groups(ssm::kSdThreads));
    if (!conv_grid(dm, conv_tokens(dm), true).fits())
        return fail(SSM_ERR_SHAPE, "batch*seqlen exceeds the convolution's launch (%lld workgroups)", (long long)max_groups(256));
    return SSM_OK;
}

// u, the rows after the last token, and with `tok` the tokens' decays
template <typename IO>
void launch_conv(const void *x_, const float *w, const float *bias, const void *st_in, void *st_out, const int32_t *lens,
                 void *u, const void *dt, const float *A, const float *dt_bias, float *tok, const ssm_ssd_conv_dims *dm,
                 int flags, hipStream_t st) {
    const int64_t stride = dm->xbc_stride ? dm->xbc_stride : row_of(dm);
    const int tt = conv_tokens(dm);
    const ConvGrid g = conv_grid(dm, tt, tok);
    const ssm::sd_tok_args k = {dt, A, dt_bias, tok, dm->dt_stride ? dm->dt_stride : dm->nheads, chunks(dm), (int)dm->nheads,
                                flags & SSM_SCAN_SOFTPLUS, (int)g.blocks};
    const bool al = aligned(x_, ssm::kSdConvV * sizeof(IO)) && stride % ssm::kSdConvV == 0;
    auto kern = dm->width == ssm::kSdTaps ? al ? ssm::sd_conv_kernel<IO, true, true> : ssm::sd_conv_kernel<IO, false, true>
              : al ? ssm::sd_conv_kernel<IO, true, false> : ssm::sd_conv_kernel<IO, false, false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(g.blocks + g.quads)), dim3(256), 0, st, static_cast<const IO *>(x_), stride, w, bias,
                       (int)dm->width, static_cast<const IO *>(st_in), static_cast<IO *>(st_out), lens, static_cast<IO *>(u),
                       dm->seqlen, (int)row_of(dm), tt, (int)g.vblocks, (int)g.tiles, k);
}

template <typename E, int NT, bool ADJ>
void launch_walk(const void *u, const void *dy, const float *tok, const int32_t *lens, const float *from, float *each, float *to,
                 int ends, const ssm_ssd_conv_dims *dm, int flags, hipStream_t st) {
    using IO = typename ssm::sd<E>::io;
    const ssm::sd_shape s = shape_of(dm, flags);
    auto kern = s.N == NT && s.P % 64 == 0 ? ssm::sd_walk_kernel<E, NT, ADJ, true> : ssm::sd_walk_kernel<E, NT, ADJ, false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(dm->batch * s.H * s.PT * s.nseg)), dim3(ssm::kSdThreads), 0,
                       st, static_cast<const IO *>(u), static_cast<const IO *>(dy), tok, lens, from, each, to, ends, s);
}
template <bool ADJ>
void walk(const void *u, const void *dy, const float *tok, const int32_t *lens, const float *from, float *each, float *to, int ends,
          const ssm_ssd_conv_dims *dm, int flags, hipStream_t st) {
    const bool bf = dm->io_dtype == SSM_IO_BF16, wide = dm->dstate > 64;
    auto f = bf ? wide ? launch_walk<__bf16, 128, ADJ> : launch_walk<__bf16, 64, ADJ>
                : wide ? launch_walk<float, 128, ADJ> : launch_walk<float, 64, ADJ>;
    f(u, dy, tok, lens, from, each, to, ends, dm, flags, st);
}

// What the segments start from: `first` where there is one, else found in `seg` by a pass over the state alone.
template <bool ADJ>
const float *segment_starts(const void *u, const void *dy, const float *tok, const int32_t *lens, const float *first, float *seg,
                            const ssm_ssd_conv_dims *dm, int flags, hipStream_t st) {
    const ssm::sd_shape s = shape_of(dm, flags);
    if (s.nseg == 1) return first;
    walk<ADJ>(u, dy, tok, lens, nullptr, nullptr, seg, 1, dm, flags, st);
    const int blocks = (int)ceil_div((int64_t)s.P * s.N, 1024);
    hipLaunchKernelGGL(ssm::sd_combine_kernel<ADJ>, dim3((unsigned)(dm->batch * s.H * blocks)), dim3(256), s.nseg * sizeof(float), st,
                       tok, first, seg, s, blocks);
    return seg;
}

template <typename E, int NT>
void launch_scan(const void *u, const float *tok, const float *D, const int32_t *lens, const float *from, void *y, float *last, float *ckpt, const ssm_ssd_conv_dims *dm, int flags, hipStream_t st) {
    using IO = typename ssm::sd<E>::io;
    const ssm::sd_shape s = shape_of(dm, flags);
    auto kern = s.N == NT && s.P % 64 == 0 ? ssm::sd_scan_kernel<E, NT, true> : ssm::sd_scan_kernel<E, NT, false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(dm->batch * s.H * s.PT * s.nseg)), dim3(ssm::kSdThreads), 0, st,
                       static_cast<const IO *>(u), tok, D, lens, from, static_cast<IO *>(y), last, ckpt, s);
}

// The step's launches (of few heads in parts there are at most 2048 and as many again).
int check_step(const ssm_ssd_conv_dims *dm) {
    const int rc = check_dims(dm);
    if (rc != SSM_OK) return rc;
    if (dm->batch > max_groups(256) / std::max(ceil_div(row_of(dm) / ssm::kSdConvV, 256), dm->nheads))
        return fail(SSM_ERR_SHAPE, "batch*nheads or batch*ceil(row/1024) exceeds %lld, the workgroups of a launch",
                    (long long)max_groups(256));
    return SSM_OK;
}

template <typename IO>
void launch_step(float *state, const void *u, const void *dt, const float *A, const float *D, const float *dt_bias, void *y,
                 const ssm_ssd_conv_dims *dm, int flags, hipStream_t st) {
    const ssm::sd_shape s = shape_of(dm, flags);
    // Lanes per channel; two channels of a thread at a time, and a head's channels in several workgroups where there
    // are few heads (one sequence of 32 heads P64 N128: 3.9 us, 6.6 with one workgroup a head)
    const int lanes = s.N / 4, lpr = lanes <= 2 ? 2 : lanes <= 4 ? 4 : lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
    const int64_t heads = dm->batch * s.H, most = ceil_div(s.P, 2 * (256 / lpr));
    const int parts = (int)std::min<int64_t>(most, std::max<int64_t>(2048 / heads, 1));
    auto kern = lpr == 2 ? ssm::sd_step_kernel<IO, 2, 2> : lpr == 4 ? ssm::sd_step_kernel<IO, 4, 2>
              : lpr == 8 ? ssm::sd_step_kernel<IO, 8, 2> : lpr == 16 ? ssm::sd_step_kernel<IO, 16, 2> : ssm::sd_step_kernel<IO, 32, 2>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(heads * parts)), dim3(256), 0, st, state, static_cast<const IO *>(u),
                       static_cast<const IO *>(dt), s.dt_stride, A, D, dt_bias, s.softplus, static_cast<IO *>(y), s.H, s.P,
                       s.G, s.N, parts);
}

template <typename IO>
void launch_conv_step(const void *x_, const float *w, const float *bias, void *st_rows, void *u, const ssm_ssd_conv_dims *dm,
                      hipStream_t st) {
    const int64_t stride = dm->xbc_stride ? dm->xbc_stride : row_of(dm), vblocks = ceil_div(row_of(dm) / ssm::kSdConvV, 256);
    const bool al = aligned(x_, ssm::kSdConvV * sizeof(IO)) && stride % ssm::kSdConvV == 0;
    auto kern = al ? ssm::sd_conv_step_kernel<IO, true> : ssm::sd_conv_step_kernel<IO, false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(vblocks * dm->batch)), dim3(256), 0, st, static_cast<const IO *>(x_), stride, w, bias,
                       (int)dm->width, static_cast<IO *>(st_rows), static_cast<IO *>(u), (int)row_of(dm), (int)vblocks);
}

// How the backward cuts its work, and its workspace.
// Tokens per thread of the convolution's backward: 64 (a thread goes three tokens further than its own), 16 where
// that leaves CUs with less than four waves per SIMD (B5 L777 of 2,304 channels bf16: 20 us with 16, 33 with 64; B2
// L2048 of 1,664 fp32: 20 and 40; B8 L2048 of 5,248 bf16: 163 and 149).
int conv_bwd_tokens(const ssm_ssd_conv_dims *dm) {
    return dm->batch * dm->seqlen * (row_of(dm) / ssm::kSdConvV) >= (int64_t)64 * 64 * 4096 ? 64 : 16;
}
struct BwdPlan {
    int HS, hpw;
    int64_t tiles;
    size_t u, tok, states, seg, adjoints, du, dbc, part, conv_part, bytes;   // offsets (u, tok, states: without checkpoints)
};
BwdPlan bwd_plan(const ssm_ssd_conv_dims *dm, bool have_checkpoints) {
    BwdPlan p;
    const int64_t per = dm->nheads / dm->ngroups, items = std::max<int64_t>(dm->batch * chunks(dm) * dm->ngroups, 1);
    // Parts of a group's heads: what takes the fewest rounds of a workgroup per CU, a workgroup's start and end
    // counted as kStart heads (and its part of dB and dC written and read again).  B5 L777 G4 of five heads each: 103 us
    // in one part, 130 + 15 in five, as 0 would have it; 8 chooses as 3 does there.  (B8 L2048 H80 and B2 L2048 H24 take the
    // same time with 0, 3 and 8.)
    constexpr int64_t kCUs = 256, kStart = 3;
    int64_t best = -1;
    for (int64_t parts = 1; parts <= per; ++parts) {
        const int64_t hpw = ceil_div(per, parts), hs = ceil_div(per, hpw), cost = ceil_div(items * hs, kCUs) * (hpw + kStart);
        if (best < 0 || cost < best) {
            best = cost;
            p.hpw = (int)hpw;
            p.HS = (int)hs;
        }
        if (items * hs > 8 * kCUs) break;
    }
    p.tiles = std::max<int64_t>(ceil_div(dm->seqlen, conv_bwd_tokens(dm)), 1);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += align256(bytes);
        return o;
    };
    const size_t tokens = (size_t)(dm->batch * dm->seqlen);
    p.u = take(have_checkpoints ? 0 : u_bytes(dm));
    p.tok = take(have_checkpoints ? 0 : tok_bytes(dm));
    p.states = take(have_checkpoints ? 0 : state_bytes(dm));
    p.seg = take(seg_bytes(dm));
    p.adjoints = take(state_bytes(dm));
    p.du = take(tokens * dm->nheads * dm->headdim * 4);
    p.dbc = take(tokens * p.HS * 2 * dm->ngroups * dm->dstate * 4);
    p.part = take((size_t)(dm->batch * chunks(dm) * 3 * dm->nheads) * 4);
    p.conv_part = take((size_t)(dm->batch * p.tiles * 5 * row_of(dm)) * 4);
    p.bytes = at;
    return p;
}

// The backward's launches (those of a forward among them, which forms what there are no checkpoints of).
int check_backward(const ssm_ssd_conv_dims *dm, int flags) {
    const int rc = check_forward(dm);
    if (rc != SSM_OK || dm->batch == 0 || dm->nheads == 0) return rc;
    if (dm->batch * chunks(dm) > max_groups(ssm::kSdBwdThreads) / (dm->ngroups * bwd_plan(dm, flags & SSM_SCAN_CHECKPOINTS).HS))
        return fail(SSM_ERR_SHAPE, "batch*ceil(seqlen/64)*ngroups exceeds the backward's launch (%lld workgroups)",
                    (long long)max_groups(ssm::kSdBwdThreads));
    if (!conv_grid(dm, conv_bwd_tokens(dm), false).fits())
        return fail(SSM_ERR_SHAPE, "batch*seqlen exceeds the launch of the convolution's backward (%lld workgroups)",
                    (long long)max_groups(256));
    return SSM_OK;   // (there are parts of a group's heads for few items only: their sums are of at most 2^25 elements)
}

template <typename E, int NT>
void launch_bwd(const void *u, const void *dy, const float *tok, const void *dt, const float *A, const float *D, const float *dt_bias,
                const int32_t *lens, const float *states, const float *adjoints, void *ddt, const ssm::sd_grad &g,
                const ssm_ssd_conv_dims *dm, int flags, hipStream_t st) {
    using IO = typename ssm::sd<E>::io;
    const ssm::sd_shape s = shape_of(dm, flags);
    auto kern = s.N == 64 && s.P == 64 ? ssm::sd_bwd_kernel<E, NT, NT == 64 ? 2 : 1>
              : s.N == NT && s.P % 64 == 0 ? ssm::sd_bwd_kernel<E, NT, 1> : ssm::sd_bwd_kernel<E, NT, 0>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(dm->batch * s.nchunk * s.G * g.HS)), dim3(ssm::kSdBwdThreads), 0, st,
                       static_cast<const IO *>(u), static_cast<const IO *>(dy), tok, static_cast<const IO *>(dt), A, D, dt_bias, lens,
                       states, adjoints, static_cast<IO *>(ddt), g, s);
}

template <typename IO>
void launch_conv_bwd(const void *x_, const float *w, const float *bias, const void *st_in, const int32_t *lens, const float *du,
                     const float *dbc, void *dx, void *dst, float *parts, const ssm_ssd_conv_dims *dm, hipStream_t st) {
    const int64_t stride = dm->xbc_stride ? dm->xbc_stride : row_of(dm);
    const ConvGrid g = conv_grid(dm, conv_bwd_tokens(dm), false);
    const bool al = aligned(x_, ssm::kSdConvV * sizeof(IO)) && stride % ssm::kSdConvV == 0;
    auto kern = dm->width == ssm::kSdTaps ? al ? ssm::sd_conv_bwd_kernel<IO, true, true> : ssm::sd_conv_bwd_kernel<IO, false, true>
              : al ? ssm::sd_conv_bwd_kernel<IO, true, false> : ssm::sd_conv_bwd_kernel<IO, false, false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)g.blocks), dim3(256), 0, st, static_cast<const IO *>(x_), stride, w, bias,
                       (int)dm->width, static_cast<const IO *>(st_in), lens, du, dbc, static_cast<IO *>(dx),
                       static_cast<IO *>(dst), parts, dm->seqlen, (int)row_of(dm), (int)(dm->nheads * dm->headdim),
                       conv_bwd_tokens(dm), (int)g.vblocks, (int)g.tiles);
}

void launch_sums(const float *part, int64_t n, int cols, int planes, const ssm::sd_sums &o, hipStream_t st) {
    const int blocks = (cols + ssm::kSdSumCols - 1) / ssm::kSdSumCols * planes;
    hipLaunchKernelGGL(ssm::sd_sum_kernel, dim3((unsigned)blocks), dim3(ssm::kSdSumCols * ssm::kSdSumGroups), 0, st, part, n, cols,
                       planes, o);
}

int check_workspace(const void *ws, size_t have, size_t need) {
    if (need > 0 && !ws) return fail(SSM_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (have < need) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", have, need);
    if (need > 0 && !aligned(ws, 16)) return fail(SSM_ERR_ALIGN, "workspace not 16-byte aligned");
    return SSM_OK;
}

}  // namespace

extern "C" {

size_t ssm_ssd_conv_workspace_bytes(const ssm_ssd_conv_dims *dims, int flags) {
    if (check_forward(dims) != SSM_OK || dims->batch == 0 || dims->nheads == 0) return 0;
    return u_bytes(dims) + tok_bytes(dims) + ((flags & SSM_SCAN_CHECKPOINTS) ? state_bytes(dims) : 0) + seg_bytes(dims);
}

int ssm_ssd_conv_fwd(const void *xbc, const float *conv_w, const float *conv_b, const void *conv_state, const void *dt,
                     const float *A, const float *D, const float *dt_bias, const float *initial_state,
                     const int32_t *seq_lens, int flags, void *y, float *last_state, void *conv_state_out,
                     const ssm_ssd_conv_dims *dims, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_forward(dims);
    if (rc != SSM_OK) return rc;
    if (flags & ~(SSM_SCAN_SOFTPLUS | SSM_SCAN_CHECKPOINTS)) return fail(SSM_ERR_FLAGS, "unknown flag bits 0x%x", flags);
    const size_t es = elem_size(dims);
    if (!aligned(xbc, es) || !aligned(dt, es) || !aligned(conv_w, 4) || !aligned(conv_b, 4) || !aligned(A, 4) || !aligned(D, 4) ||
        !aligned(dt_bias, 4) || !aligned(seq_lens, 4))
        return fail(SSM_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    if (!aligned(y, 16) || !aligned(initial_state, 16) || !aligned(last_state, 16) || !aligned(conv_state, 16) ||
        !aligned(conv_state_out, 16))
        return fail(SSM_ERR_ALIGN, "y, the states or the convolution's rows are not 16-byte aligned");
    if (dims->batch == 0 || dims->nheads == 0) return ok();
    if (!conv_w || !A) return fail(SSM_ERR_NULL, "conv_w or A is NULL");
    if (dims->seqlen > 0 && (!xbc || !dt || !y)) return fail(SSM_ERR_NULL, "xbc, dt or y is NULL");
    rc = check_workspace(workspace, workspace_bytes, ssm_ssd_conv_workspace_bytes(dims, flags));
    if (rc != SSM_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    float *tok = reinterpret_cast<float *>(static_cast<char *>(workspace) + u_bytes(dims));
    float *ckpt = (flags & SSM_SCAN_CHECKPOINTS) ? tok + tok_bytes(dims) / sizeof(float) : nullptr;
    const bool bf = es == 2, wide = dims->dstate > 64;
    auto conv = bf ? launch_conv<uint16_t> : launch_conv<float>;
    conv(xbc, conv_w, conv_b, conv_state, conv_state_out, seq_lens, workspace, dt, A, dt_bias, tok, dims, flags, st);
    auto scan = bf ? wide ? launch_scan<__bf16, 128> : launch_scan<__bf16, 64> : wide ? launch_scan<float, 128> : launch_scan<float, 64>;
    float *seg = tok + (tok_bytes(dims) + (ckpt ? state_bytes(dims) : 0)) / sizeof(float);
    const float *from = segment_starts<false>(workspace, nullptr, tok, seq_lens, initial_state, seg, dims, flags, st);
    scan(workspace, tok, D, seq_lens, from, y, last_state, ckpt, dims, flags, st);
    return launched();
}

size_t ssm_ssd_conv_bwd_workspace_bytes(const ssm_ssd_conv_dims *dims, int flags) {
    if (check_backward(dims, flags) != SSM_OK || dims->batch == 0 || dims->nheads == 0) return 0;
    return bwd_plan(dims, flags & SSM_SCAN_CHECKPOINTS).bytes;
}

int ssm_ssd_conv_bwd(const void *xbc, const float *conv_w, const float *conv_b, const void *conv_state, const void *dt,
                     const float *A, const float *D, const float *dt_bias, const float *initial_state,
                     const int32_t *seq_lens, int flags, const void *dy, const float *dlast_state, const void *checkpoints,
                     size_t checkpoints_bytes, void *dxbc, float *dconv_w, float *dconv_b, void *dconv_state, void *ddt,
                     float *dA, float *dD, float *ddt_bias, float *dinitial_state, const ssm_ssd_conv_dims *dims,
                     void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_backward(dims, flags);
    if (rc != SSM_OK) return rc;
    if (flags & ~(SSM_SCAN_SOFTPLUS | SSM_SCAN_CHECKPOINTS)) return fail(SSM_ERR_FLAGS, "unknown flag bits 0x%x", flags);
    const size_t es = elem_size(dims);
    if (!aligned(xbc, es) || !aligned(dt, es) || !aligned(ddt, es) || !aligned(conv_w, 4) || !aligned(conv_b, 4) || !aligned(A, 4) ||
        !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(seq_lens, 4) || !aligned(dconv_w, 4) || !aligned(dconv_b, 4) ||
        !aligned(dA, 4) || !aligned(dD, 4) || !aligned(ddt_bias, 4))
        return fail(SSM_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    if (!aligned(dy, 16) || !aligned(dxbc, 16) || !aligned(initial_state, 16) || !aligned(dlast_state, 16) ||
        !aligned(dinitial_state, 16) || !aligned(conv_state, 16) || !aligned(dconv_state, 16) || !aligned(checkpoints, 16))
        return fail(SSM_ERR_ALIGN, "dy, dxbc, the states, the convolution's rows or the checkpoints are not 16-byte aligned");
    if (dims->nheads == 0) return ok();
    if (!conv_w || !A || !dconv_w || !dA) return fail(SSM_ERR_NULL, "conv_w, A, dconv_w or dA is NULL");
    if (dims->batch > 0 && dims->seqlen > 0 && (!xbc || !dt || !dy || !dxbc || !ddt))
        return fail(SSM_ERR_NULL, "xbc, dt, dy, dxbc or ddt is NULL");
    const bool kept = flags & SSM_SCAN_CHECKPOINTS;
    if (kept) {
        const size_t need = ssm_ssd_conv_workspace_bytes(dims, SSM_SCAN_CHECKPOINTS);
        if (need > 0 && !checkpoints) return fail(SSM_ERR_NULL, "checkpoints is NULL with SSM_SCAN_CHECKPOINTS");
        if (checkpoints_bytes < need)
            return fail(SSM_ERR_WORKSPACE, "checkpoints of %zu bytes are smaller than the %zu of the forward", checkpoints_bytes, need);
    }
    rc = check_workspace(workspace, workspace_bytes, ssm_ssd_conv_bwd_workspace_bytes(dims, flags));
    if (rc != SSM_OK) return rc;
    const BwdPlan p = bwd_plan(dims, kept);
    hipStream_t st = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    auto at = [&](size_t o) { return reinterpret_cast<float *>(ws + o); };
    const char *ck = static_cast<const char *>(checkpoints);
    const void *u = kept ? ck : ws + p.u;
    const float *tok = kept ? reinterpret_cast<const float *>(ck + u_bytes(dims)) : at(p.tok);
    const float *states = kept ? tok + tok_bytes(dims) / sizeof(float) : at(p.states);
    const bool bf = es == 2, wide = dims->dstate > 64;
    if (dims->batch > 0) {
        if (!kept) {
            auto conv = bf ? launch_conv<uint16_t> : launch_conv<float>;
            conv(xbc, conv_w, conv_b, conv_state, nullptr, seq_lens, ws + p.u, dt, A, dt_bias, at(p.tok), dims, flags, st);
            const float *from = segment_starts<false>(u, nullptr, tok, seq_lens, initial_state, at(p.seg), dims, flags, st);
            walk<false>(u, nullptr, tok, seq_lens, from, at(p.states), nullptr, 0, dims, flags, st);
        }
        const float *from = segment_starts<true>(u, dy, tok, seq_lens, dlast_state, at(p.seg), dims, flags, st);
        walk<true>(u, dy, tok, seq_lens, from, at(p.adjoints), dinitial_state, 0, dims, flags, st);
        if (dims->seqlen > 0) {
            const ssm::sd_grad g = {at(p.du), at(p.dbc), at(p.part), p.HS, p.hpw};
            auto k = bf ? wide ? launch_bwd<__bf16, 128> : launch_bwd<__bf16, 64> : wide ? launch_bwd<float, 128> : launch_bwd<float, 64>;
            k(u, dy, tok, dt, A, D, dt_bias, seq_lens, states, at(p.adjoints), ddt, g, dims, flags, st);
        }
        const int64_t nbc = dims->batch * dims->seqlen * 2 * dims->ngroups * dims->dstate;
        if (p.HS > 1 && nbc > 0)
            hipLaunchKernelGGL(ssm::sd_parts_kernel, dim3((unsigned)ceil_div(nbc, 1024)), dim3(256), 0, st, at(p.dbc), nbc, p.HS);
        auto c = bf ? launch_conv_bwd<uint16_t> : launch_conv_bwd<float>;
        c(xbc, conv_w, conv_b, conv_state, seq_lens, at(p.du), at(p.dbc), dxbc, dconv_state, at(p.conv_part), dims, st);
    }
    const int W = dims->width, H = (int)dims->nheads;
    ssm::sd_sums o = {};
    for (int j = 0; j < ssm::kSdTaps; ++j) {
        const int tap = j - (ssm::kSdTaps - W);
        o.out[j] = tap >= 0 ? dconv_w + tap : nullptr;
        o.stride[j] = W;
    }
    o.out[4] = dconv_b;
    o.stride[4] = 1;
    launch_sums(at(p.conv_part), dims->batch * p.tiles, (int)row_of(dims), 5, o, st);
    const ssm::sd_sums h = {{dA, ddt_bias, dD}, {1, 1, 1}};
    launch_sums(at(p.part), dims->batch * chunks(dims), H, 3, h, st);
    return launched();
}

size_t ssm_ssd_conv_step_workspace_bytes(const ssm_ssd_conv_dims *dims) {
    if (check_step(dims) != SSM_OK) return 0;
    return align256((size_t)(dims->batch * row_of(dims)) * elem_size(dims));
}

int ssm_ssd_conv_step(float *state, void *conv_state, const void *xbc, const float *conv_w, const float *conv_b,
                      const void *dt, const float *A, const float *D, const float *dt_bias, int flags, void *y,
                      const ssm_ssd_conv_dims *dims, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_step(dims);
    if (rc != SSM_OK) return rc;
    if (flags & ~SSM_SCAN_SOFTPLUS) return fail(SSM_ERR_FLAGS, "unknown flag bits 0x%x", flags);
    const size_t es = elem_size(dims);
    if (!aligned(xbc, es) || !aligned(dt, es) || !aligned(y, es) || !aligned(conv_w, 4) || !aligned(conv_b, 4) || !aligned(A, 4) ||
        !aligned(D, 4) || !aligned(dt_bias, 4))
        return fail(SSM_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    if (!aligned(state, 16) || !aligned(conv_state, 16))
        return fail(SSM_ERR_ALIGN, "the state or the convolution's rows are not 16-byte aligned");
    if (dims->batch == 0 || dims->nheads == 0) return ok();
    if (!state || !xbc || !conv_w || !dt || !A || !y || (dims->width > 1 && !conv_state))
        return fail(SSM_ERR_NULL, "required pointer is NULL");
    rc = check_workspace(workspace, workspace_bytes, ssm_ssd_conv_step_workspace_bytes(dims));
    if (rc != SSM_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    ssm_ssd_conv_dims one = *dims;
    one.seqlen = 1;
    if (es == 2) {
        launch_conv_step<uint16_t>(xbc, conv_w, conv_b, conv_state, workspace, &one, st);
        launch_step<uint16_t>(state, workspace, dt, A, D, dt_bias, y, &one, flags, st);
    } else {
        launch_conv_step<float>(xbc, conv_w, conv_b, conv_state, workspace, &one, st);
        launch_step<float>(state, workspace, dt, A, D, dt_bias, y, &one, flags, st);
    }
    return launched();
}

}  // extern "C"
