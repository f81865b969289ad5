// C ABI of windowed attention and its resident cache: argument validation and
// workspace sizing.  Declarations and the full contract are in include/gdn.h.
// Every check runs before anything is enqueued.
#include "gdn.h"
#include "gdn_check.h"
#include "gdn_swa.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

namespace {

using namespace gdn;

gdn_status check_heads(int32_t heads, int32_t kv_heads) {
    if (heads < 1 || kv_heads < 1 || heads % kv_heads)
        return fail(GDN_ERR_SHAPE, "need heads >= 1 a multiple of kv_heads >= 1 (got %d, %d)", heads, kv_heads);
    if (heads > 1024 || heads / kv_heads > kSwaMaxGroup)
        return fail(GDN_ERR_UNSUPPORTED, "heads %d on kv_heads %d not built (at most 1024, at most %d a key head)", heads,
                    kv_heads, kSwaMaxGroup);
    return GDN_OK;
}

gdn_status check_swa_desc(const gdn_swa_desc *d, bool bwd) {
    if (!d) return fail(GDN_ERR_NULL, "desc is NULL");
    if (!valid_dtype(d->dtype)) return fail(GDN_ERR_DTYPE, "unknown dtype code %d", d->dtype);
    if (d->batch < 1 || d->seqlen < 0 || d->keylen < 0 || d->num_seqs < 1 || d->window < 1 || d->sinks < 0)
        return fail(GDN_ERR_SHAPE, "need batch >= 1, seqlen >= 0, keylen >= 0, num_seqs >= 1, window >= 1, sinks >= 0 "
                    "(got %d, %d, %d, %d, %d, %d)", d->batch, d->seqlen, d->keylen, d->num_seqs, d->window, d->sinks);
    if ((int64_t)d->batch * d->seqlen >= (1 << 30) || (int64_t)d->batch * d->keylen >= (1 << 30))
        return fail(GDN_ERR_SHAPE, "batch * seqlen or batch * keylen too large");
    gdn_status s = check_heads(d->heads, d->kv_heads);
    if (s != GDN_OK) return s;
    const int most = bwd || d->dtype == GDN_FP32 ? 128 : 256;
    if (!(d->dim == 32 || d->dim == 64 || d->dim == 128 || d->dim == 256) || d->dim > most)
        return fail(GDN_ERR_UNSUPPORTED, "dim %d not built here (32, 64, 128%s)", d->dim, most == 256 ? ", 256" : "");
    if (d->sinks > kSwaMaxSinks)
        return fail(GDN_ERR_UNSUPPORTED, "sinks %d not built (at most %d)", d->sinks, kSwaMaxSinks);
    if (!(std::isfinite(d->scale) && d->scale > 0.f)) return fail(GDN_ERR_UNSUPPORTED, "scale must be finite and > 0");
    if (d->flags) return fail(GDN_ERR_UNSUPPORTED, "unknown flags 0x%x", d->flags);
    return GDN_OK;
}

SwaArgs swa_args(const gdn_swa_desc &d) {
    SwaArgs a{};
    a.B = d.batch, a.T = d.seqlen, a.Tk = d.keylen, a.N = d.num_seqs, a.H = d.heads, a.KV = d.kv_heads, a.D = d.dim;
    // positions are below 2^30: a longer window sees as much, and sums with it stay in 32 bits
    a.window = std::min(d.window, 1 << 30), a.sinks = d.sinks, a.dtype = d.dtype, a.scale = d.scale;
    return a;
}

gdn_status check_swa_layout(const gdn_swa_desc &d, const int32_t *cu, const int32_t *cuk, const void *workspace,
                            size_t workspace_bytes, size_t need) {
    if (!cu != !cuk) return fail(GDN_ERR_NULL, "cu_seqlens and cu_seqlens_k are given together or not at all");
    if (cu && d.batch != 1) return fail(GDN_ERR_SHAPE, "cu_seqlens requires batch == 1 (got %d)", d.batch);
    if (!cu && d.num_seqs != d.batch)
        return fail(GDN_ERR_SHAPE, "without cu_seqlens num_seqs must equal batch (%d != %d)", d.num_seqs, d.batch);
    if (!workspace) return fail(GDN_ERR_WORKSPACE, "workspace is NULL");
    if (workspace_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace has %zu bytes, this call needs %zu", workspace_bytes, need);
    return GDN_OK;
}

gdn_status swa_size(const gdn_swa_desc *desc, size_t *bytes, bool bwd) {
    if (!bytes) return fail(GDN_ERR_NULL, "bytes is NULL");
    gdn_status s = check_swa_desc(desc, bwd);
    if (s != GDN_OK) return s;
    *bytes = swa_workspace_layout(swa_args(*desc), bwd).total;
    return ok();
}

}  // namespace

extern "C" {

gdn_status gdn_swa_fwd_workspace_size(const gdn_swa_desc *desc, size_t *bytes) { return swa_size(desc, bytes, false); }
gdn_status gdn_swa_bwd_workspace_size(const gdn_swa_desc *desc, size_t *bytes) { return swa_size(desc, bytes, true); }

gdn_status gdn_swa_fwd(const gdn_swa_desc *desc, const void *q, const void *k, const void *v,
                       const int32_t *cu_seqlens, const int32_t *cu_seqlens_k, void *o, float *lse, void *workspace,
                       size_t workspace_bytes, hipStream_t stream) {
    gdn_status s = check_swa_desc(desc, false);
    if (s != GDN_OK) return s;
    const gdn_swa_desc &d = *desc;
    SwaArgs a = swa_args(d);
    const size_t need = swa_workspace_layout(a, false).total;
    s = check_swa_layout(d, cu_seqlens, cu_seqlens_k, workspace, workspace_bytes, need);
    if (s != GDN_OK) return s;
    const size_t rows = (size_t)d.batch * d.seqlen * d.heads, keys = (size_t)d.batch * d.keylen * d.kv_heads;
    const size_t row = (size_t)d.dim * dtype_size(d.dtype), offs = 4 * ((size_t)d.num_seqs + 1);
    const Arg args[] = {{"q", q, rows * row, rows > 0, false, 16},
                        {"k", k, keys * row, keys > 0, false, 16},
                        {"v", v, keys * row, keys > 0, false, 16},
                        {"cu_seqlens", cu_seqlens, offs, false, false, 4},
                        {"cu_seqlens_k", cu_seqlens_k, offs, false, false, 4},
                        {"o", o, rows * row, rows > 0, true, 16},
                        {"lse", lse, rows * 4, false, true, 4},
                        {"workspace", workspace, need, true, true, 16}};
    s = check_args(args, 8);
    if (s == GDN_OK) s = check_overlap(args, 8);
    if (s != GDN_OK) return s;
    a.q = q, a.k = k, a.v = v, a.cu = cu_seqlens, a.cuk = cu_seqlens_k, a.o = o, a.lse = lse, a.workspace = workspace;
    hipError_t err = launch_swa_fwd(a, stream);
    if (err != hipSuccess) return hip_fail(err, "gdn_swa_fwd launch");
    return ok();
}

gdn_status gdn_swa_bwd(const gdn_swa_desc *desc, const void *d_o, const void *q, const void *k, const void *v,
                       const void *o, const float *lse, const int32_t *cu_seqlens, const int32_t *cu_seqlens_k,
                       void *dq, void *dk, void *dv, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    gdn_status s = check_swa_desc(desc, true);
    if (s != GDN_OK) return s;
    const gdn_swa_desc &d = *desc;
    SwaArgs a = swa_args(d);
    const size_t need = swa_workspace_layout(a, true).total;
    s = check_swa_layout(d, cu_seqlens, cu_seqlens_k, workspace, workspace_bytes, need);
    if (s != GDN_OK) return s;
    const size_t rows = (size_t)d.batch * d.seqlen * d.heads, keys = (size_t)d.batch * d.keylen * d.kv_heads;
    const size_t row = (size_t)d.dim * dtype_size(d.dtype), offs = 4 * ((size_t)d.num_seqs + 1);
    const Arg args[] = {{"d_o", d_o, rows * row, rows > 0, false, 16},
                        {"q", q, rows * row, rows > 0, false, 16},
                        {"k", k, keys * row, keys > 0, false, 16},
                        {"v", v, keys * row, keys > 0, false, 16},
                        {"o", o, rows * row, rows > 0, false, 16},
                        {"lse", lse, rows * 4, rows > 0, false, 4},
                        {"cu_seqlens", cu_seqlens, offs, false, false, 4},
                        {"cu_seqlens_k", cu_seqlens_k, offs, false, false, 4},
                        {"dq", dq, rows * row, rows > 0, true, 16},
                        {"dk", dk, keys * row, keys > 0, true, 16},
                        {"dv", dv, keys * row, keys > 0, true, 16},
                        {"workspace", workspace, need, true, true, 16}};
    s = check_args(args, 12);
    if (s == GDN_OK) s = check_overlap(args, 12);
    if (s != GDN_OK) return s;
    a.q = q, a.k = k, a.v = v, a.cu = cu_seqlens, a.cuk = cu_seqlens_k;
    a.o = const_cast<void *>(o), a.lse = const_cast<float *>(lse), a.d_o = d_o;
    a.dq = dq, a.dk = dk, a.dv = dv, a.workspace = workspace;
    hipError_t err = launch_swa_bwd(a, stream);
    if (err != hipSuccess) return hip_fail(err, "gdn_swa_bwd launch");
    return ok();
}

}  // extern "C"
