// C ABI of the gated linear recurrence, layer norm and the state moves:
// argument validation and workspace sizing.  Declarations and the full
// contract are in include/gdn.h.  Every check runs before anything is
// enqueued.
#include "gdn.h"
#include "gdn_check.h"
#include "gdn_ops.h"

#include <hip/hip_runtime.h>

#include <cmath>

namespace {

using namespace gdn;

gdn_status check_scan_desc(const gdn_scan_desc *d) {
    if (!d) return fail(GDN_ERR_NULL, "desc is NULL");
    const int32_t dt[] = {d->in_dtype, d->gate_dtype, d->out_dtype};
    gdn_status s = check_types(dt, 3);
    if (s != GDN_OK) return s;
    if (d->batch < 1 || d->seqlen < 0 || d->channels < 1 || d->num_seqs < 1)
        return fail(GDN_ERR_SHAPE, "need batch >= 1, seqlen >= 0, channels >= 1, num_seqs >= 1 (got %d, %d, %d, %d)",
                    d->batch, d->seqlen, d->channels, d->num_seqs);
    if ((int64_t)d->batch * d->seqlen >= (1 << 30)) return fail(GDN_ERR_SHAPE, "batch * seqlen too large");
    if (d->channels > 65536) return fail(GDN_ERR_UNSUPPORTED, "channels %d not built (at most 65536)", d->channels);
    if (d->flags) return fail(GDN_ERR_UNSUPPORTED, "unknown flags 0x%x", d->flags);
    return GDN_OK;
}

gdn_status check_scan_layout(const gdn_scan_desc &d, bool packed, const void *workspace, size_t workspace_bytes,
                             size_t need) {
    if (packed && d.batch != 1) return fail(GDN_ERR_SHAPE, "cu_seqlens requires batch == 1 (got %d)", d.batch);
    if (!packed && d.num_seqs != d.batch)
        return fail(GDN_ERR_SHAPE, "without cu_seqlens num_seqs must equal batch (%d != %d)", d.num_seqs, d.batch);
    if (!workspace) return fail(GDN_ERR_WORKSPACE, "workspace is NULL");
    if (workspace_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace has %zu bytes, this call needs %zu", workspace_bytes, need);
    return GDN_OK;
}

gdn_status check_norm(int64_t rows, int32_t dim) {
    if (rows < 0 || rows > INT32_MAX || dim < 1)
        return fail(GDN_ERR_SHAPE, "need 0 <= rows < 2^31 and dim >= 1 (got %lld, %d)", (long long)rows, dim);
    if (dim > kNormMaxDim) return fail(GDN_ERR_UNSUPPORTED, "dim %d not built (at most %d)", dim, kNormMaxDim);
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_scan_workspace_size(const gdn_scan_desc *desc, size_t *bytes) {
    if (!bytes) return fail(GDN_ERR_NULL, "bytes is NULL");
    gdn_status s = check_scan_desc(desc);
    if (s != GDN_OK) return s;
    // The larger of the packed and the batched layout: the answer does not
    // depend on whether cu_seqlens is passed later.
    const auto a = scan_workspace_layout(desc->batch, desc->seqlen, desc->channels, desc->num_seqs, true);
    const auto b = scan_workspace_layout(desc->batch, desc->seqlen, desc->channels, desc->num_seqs, false);
    *bytes = a.total > b.total ? a.total : b.total;
    return ok();
}

gdn_status gdn_scan_fwd(const gdn_scan_desc *desc, const void *x, const void *log_alpha, const float *init_state,
                        const int32_t *cu_seqlens, void *h, float *final_state, void *workspace,
                        size_t workspace_bytes, hipStream_t stream) {
    gdn_status s = check_scan_desc(desc);
    if (s != GDN_OK) return s;
    const gdn_scan_desc &d = *desc;
    const bool packed = cu_seqlens != nullptr;
    const auto w = scan_workspace_layout(d.batch, d.seqlen, d.channels, d.num_seqs, packed);
    s = check_scan_layout(d, packed, workspace, workspace_bytes, w.total);
    if (s != GDN_OK) return s;
    const size_t e = (size_t)d.batch * d.seqlen * d.channels, st = (size_t)d.num_seqs * d.channels * 4;
    const bool some = e > 0;
    const Arg args[] = {{"x", x, e * dtype_size(d.in_dtype), some, false, 16},
                        {"log_alpha", log_alpha, e * dtype_size(d.gate_dtype), some, false, 16},
                        {"init_state", init_state, st, false, false, 16},
                        {"cu_seqlens", cu_seqlens, 4 * ((size_t)d.num_seqs + 1), false, false, 4},
                        {"h", h, e * dtype_size(d.out_dtype), some, true, 16},
                        {"final_state", final_state, st, false, true, 16},
                        {"workspace", workspace, w.total, true, true, 16}};
    s = check_args(args, 7);
    if (s == GDN_OK) s = check_overlap(args, 7, 2, 5);
    if (s != GDN_OK) return s;
    ScanArgs a{};
    a.B = d.batch, a.T = d.seqlen, a.D = d.channels, a.N = d.num_seqs;
    a.in_dtype = d.in_dtype, a.gate_dtype = d.gate_dtype, a.out_dtype = d.out_dtype;
    a.x = x, a.log_alpha = log_alpha, a.init_state = init_state, a.cu_seqlens = cu_seqlens;
    a.h = h, a.final_state = final_state, a.workspace = workspace;
    hipError_t err = launch_scan_fwd(a, stream);
    if (err != hipSuccess) return hip_fail(err, "gdn_scan_fwd launch");
    return ok();
}

gdn_status gdn_scan_bwd(const gdn_scan_desc *desc, const void *log_alpha, const void *h, const float *init_state,
                        const int32_t *cu_seqlens, const void *d_h, const float *d_final_state, void *dx,
                        void *dlog_alpha, float *d_init_state, void *workspace, size_t workspace_bytes,
                        hipStream_t stream) {
    gdn_status s = check_scan_desc(desc);
    if (s != GDN_OK) return s;
    const gdn_scan_desc &d = *desc;
    const bool packed = cu_seqlens != nullptr;
    const auto w = scan_workspace_layout(d.batch, d.seqlen, d.channels, d.num_seqs, packed);
    s = check_scan_layout(d, packed, workspace, workspace_bytes, w.total);
    if (s != GDN_OK) return s;
    const size_t e = (size_t)d.batch * d.seqlen * d.channels, st = (size_t)d.num_seqs * d.channels * 4;
    const bool some = e > 0;
    const Arg args[] = {{"log_alpha", log_alpha, e * dtype_size(d.gate_dtype), some, false, 16},
                        {"h", h, e * dtype_size(d.out_dtype), some, false, 16},
                        {"init_state", init_state, st, false, false, 16},
                        {"cu_seqlens", cu_seqlens, 4 * ((size_t)d.num_seqs + 1), false, false, 4},
                        {"d_h", d_h, e * dtype_size(d.out_dtype), some, false, 16},
                        {"d_final_state", d_final_state, st, false, false, 16},
                        {"dx", dx, e * dtype_size(d.in_dtype), some, true, 16},
                        {"dlog_alpha", dlog_alpha, e * dtype_size(d.gate_dtype), some, true, 16},
                        {"d_init_state", d_init_state, st, false, true, 16},
                        {"workspace", workspace, w.total, true, true, 16}};
    s = check_args(args, 10);
    if (s == GDN_OK) s = check_overlap(args, 10);
    if (s != GDN_OK) return s;
    ScanArgs a{};
    a.B = d.batch, a.T = d.seqlen, a.D = d.channels, a.N = d.num_seqs;
    a.in_dtype = d.in_dtype, a.gate_dtype = d.gate_dtype, a.out_dtype = d.out_dtype;
    a.log_alpha = log_alpha, a.init_state = init_state, a.cu_seqlens = cu_seqlens;
    a.h = const_cast<void *>(h), a.d_h = d_h, a.d_final = d_final_state;
    a.dx = dx, a.dlog_alpha = dlog_alpha, a.d_init = d_init_state, a.workspace = workspace;
    hipError_t err = launch_scan_bwd(a, stream);
    if (err != hipSuccess) return hip_fail(err, "gdn_scan_bwd launch");
    return ok();
}

gdn_status gdn_scan_step(int32_t N, int32_t D, int32_t in_dtype, int32_t gate_dtype, int32_t out_dtype, float *state,
                         const void *x, const void *log_alpha, void *h, hipStream_t stream) {
    const int32_t dt[] = {in_dtype, gate_dtype, out_dtype};
    gdn_status s = check_types(dt, 3);
    if (s != GDN_OK) return s;
    if (N < 0 || D < 1) return fail(GDN_ERR_SHAPE, "need N >= 0 and D >= 1 (got %d, %d)", N, D);
    if (D > 65536) return fail(GDN_ERR_UNSUPPORTED, "D %d not built (at most 65536)", D);
    const int64_t e = (int64_t)N * D;
    if (e >= ((int64_t)1 << 40)) return fail(GDN_ERR_SHAPE, "N * D too large");
    if (e == 0) return ok();
    const Arg args[] = {{"state", state, (size_t)e * 4, true, true, 16},
                        {"x", x, (size_t)e * dtype_size(in_dtype), true, false, 16},
                        {"log_alpha", log_alpha, (size_t)e * dtype_size(gate_dtype), true, false, 16},
                        {"h", h, (size_t)e * dtype_size(out_dtype), true, true, 16}};
    s = check_args(args, 4);
    if (s == GDN_OK) s = check_overlap(args, 4);
    if (s != GDN_OK) return s;
    ScanStepArgs a{N, D, in_dtype, gate_dtype, out_dtype, state, x, log_alpha, h};
    hipError_t err = launch_scan_step(a, stream);
    if (err != hipSuccess) return hip_fail(err, "gdn_scan_step launch");
    return ok();
}

gdn_status gdn_layernorm_fwd(int64_t rows, int32_t dim, int32_t in_dtype, int32_t out_dtype, float eps, const void *x,
                             const float *weight, const float *bias, void *y, float *mean, float *rstd,
                             hipStream_t stream) {
    const int32_t dt[] = {in_dtype, out_dtype};
    gdn_status s = check_types(dt, 2);
    if (s == GDN_OK) s = check_norm(rows, dim);
    if (s != GDN_OK) return s;
    if (!(std::isfinite(eps) && eps >= 0.f)) return fail(GDN_ERR_UNSUPPORTED, "eps must be finite and >= 0");
    if (!mean != !rstd) return fail(GDN_ERR_NULL, "mean and rstd are returned together or not at all");
    if (rows == 0) return ok();
    const size_t e = (size_t)rows * dim, p = (size_t)dim * 4, r = (size_t)rows * 4;
    const Arg args[] = {{"x", x, e * dtype_size(in_dtype), true, false, 16},
                        {"weight", weight, p, false, false, 16},
                        {"bias", bias, p, false, false, 16},
                        {"y", y, e * dtype_size(out_dtype), true, true, 16},
                        {"mean", mean, r, false, true, 4},
                        {"rstd", rstd, r, false, true, 4}};
    s = check_args(args, 6);
    if (s == GDN_OK) s = check_overlap(args, 6);
    if (s != GDN_OK) return s;
    NormArgs a{};
    a.rows = rows, a.dim = dim, a.in_dtype = in_dtype, a.out_dtype = out_dtype, a.eps = eps;
    a.x = x, a.weight = weight, a.bias = bias, a.y = y, a.mean = mean, a.rstd = rstd;
    hipError_t err = launch_layernorm_fwd(a, stream);
    if (err != hipSuccess) return hip_fail(err, "gdn_layernorm_fwd launch");
    return ok();
}

gdn_status gdn_layernorm_bwd_workspace_size(int64_t rows, int32_t dim, size_t *bytes) {
    if (!bytes) return fail(GDN_ERR_NULL, "bytes is NULL");
    gdn_status s = check_norm(rows, dim);
    if (s != GDN_OK) return s;
    *bytes = layernorm_bwd_workspace(rows, dim);
    return ok();
}

gdn_status gdn_layernorm_bwd(int64_t rows, int32_t dim, int32_t in_dtype, int32_t out_dtype, const void *dy,
                             const void *x, const float *mean, const float *rstd, const float *weight, void *dx,
                             float *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    const int32_t dt[] = {in_dtype, out_dtype};
    gdn_status s = check_types(dt, 2);
    if (s == GDN_OK) s = check_norm(rows, dim);
    if (s != GDN_OK) return s;
    const bool sums = dweight || dbias, some = rows > 0;
    const size_t e = (size_t)rows * dim, p = (size_t)dim * 4, r = (size_t)rows * 4;
    const size_t need = sums ? layernorm_bwd_workspace(rows, dim) : 0;
    if (need && !workspace) return fail(GDN_ERR_WORKSPACE, "workspace is NULL");
    if (need && workspace_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace has %zu bytes, this call needs %zu", workspace_bytes, need);
    const Arg args[] = {{"dy", dy, e * dtype_size(out_dtype), some, false, 16},
                        {"x", x, e * dtype_size(in_dtype), some, false, 16},
                        {"mean", mean, r, some, false, 4},
                        {"rstd", rstd, r, some, false, 4},
                        {"weight", weight, p, false, false, 16},
                        {"dx", dx, e * dtype_size(in_dtype), some, true, 16},
                        {"dweight", dweight, p, false, true, 16},
                        {"dbias", dbias, p, false, true, 16},
                        {"workspace", workspace, need, false, true, 16}};
    s = check_args(args, 9);
    if (s == GDN_OK) s = check_overlap(args, 9);
    if (s != GDN_OK) return s;
    NormArgs a{};
    a.rows = rows, a.dim = dim, a.in_dtype = in_dtype, a.out_dtype = out_dtype;
    a.x = x, a.weight = weight, a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
    a.dy = dy, a.dx = dx, a.dweight = dweight, a.dbias = dbias, a.workspace = workspace;
    hipError_t err = launch_layernorm_bwd(a, stream);
    if (err != hipSuccess) return hip_fail(err, "gdn_layernorm_bwd launch");
    return ok();
}

gdn_status gdn_state_move(int32_t layers, int32_t slots, int64_t page_bytes, int32_t moves, void *state,
                          const int32_t *src, const int32_t *dst, int32_t *status, hipStream_t stream) {
    if (layers < 0 || slots < 1 || page_bytes < 4 || moves < 0 || moves > slots)
        return fail(GDN_ERR_SHAPE, "need layers >= 0, slots >= 1, page_bytes >= 4, 0 <= moves <= slots (got %d, %d, "
                    "%lld, %d)", layers, slots, (long long)page_bytes, moves);
    if (slots > kMoveMaxSlots) return fail(GDN_ERR_UNSUPPORTED, "slots %d not built (at most %d)", slots, kMoveMaxSlots);
    if (moves > kMoveMaxMoves) return fail(GDN_ERR_UNSUPPORTED, "moves %d not built (at most %d)", moves, kMoveMaxMoves);
    if (page_bytes % 4) return fail(GDN_ERR_UNSUPPORTED, "page_bytes must be a multiple of 4");
    if (page_bytes >= ((int64_t)1 << 40) || (double)layers * slots * page_bytes >= (double)((int64_t)1 << 62))
        return fail(GDN_ERR_SHAPE, "state too large");
    const size_t idx = (size_t)moves * 4;
    const bool some = moves > 0;
    const Arg args[] = {{"state", state, (size_t)layers * slots * page_bytes, some && layers > 0, true, 16},
                        {"src", src, idx, some, false, 4},
                        {"dst", dst, idx, some, false, 4},
                        {"status", status, 8, false, true, 4}};
    gdn_status s = check_args(args, 4);
    if (s == GDN_OK) s = check_overlap(args, 4);
    if (s != GDN_OK) return s;
    MoveArgs a{layers, slots, moves, page_bytes, state, src, dst, status};
    hipError_t err = launch_state_move(a, stream);
    if (err != hipSuccess) return hip_fail(err, "gdn_state_move launch");
    return ok();
}

}  // extern "C"
