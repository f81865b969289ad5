// C ABI of windowed attention and its resident cache: argument validation and
// workspace sizing.  Declarations and the full contract are in include/gdn.h.
// Every check runs before anything is enqueued.
#include "gdn.h"
#include "gdn_cache.h"
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

// Scores are taken times scale log2(e).
gdn_status check_scale(float scale) {
    if (scale > 0.f && std::isfinite(scale * 1.4426950408889634f)) return GDN_OK;
    return fail(GDN_ERR_UNSUPPORTED, "scale must be > 0 and at most 2^127");
}

SwaArgs swa_args(const gdn_swa_desc &d) {
    SwaArgs a{};
    a.B = d.batch, a.T = d.seqlen, a.Tk = d.keylen, a.N = d.num_seqs, a.H = d.heads, a.KV = d.kv_heads, a.D = d.dim;
    // positions are below 2^30: a longer window sees as much, and sums with it stay in 32 bits
    a.window = std::min(d.window, 1 << 30), a.sinks = d.sinks, a.dtype = d.dtype, a.scale = d.scale;
    return a;
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
    s = check_scale(d->scale);
    if (s != GDN_OK) return s;
    // a block for each unit and key head, two where the backward pass splits its key side
    const SwaWorkspace w = swa_workspace_layout(swa_args(*d), bwd);
    if (std::max(w.row_units, 2 * w.key_units) * (int64_t)d->kv_heads >= INT32_MAX - 7)
        return fail(GDN_ERR_SHAPE, "too many sequences, tokens and kv_heads");
    if (d->flags) return fail(GDN_ERR_UNSUPPORTED, "unknown flags 0x%x", d->flags);
    return GDN_OK;
}

// need: 0 where no workspace is read.
gdn_status check_swa_layout(const gdn_swa_desc &d, const int32_t *cu, const int32_t *cuk, const void *workspace,
                            size_t workspace_bytes, size_t need) {
    if (!cu != !cuk) return fail(GDN_ERR_NULL, "cu_seqlens and cu_seqlens_k are given together or not at all");
    if (cu && d.batch != 1) return fail(GDN_ERR_SHAPE, "cu_seqlens requires batch == 1 (got %d)", d.batch);
    if (!cu && d.num_seqs != d.batch)
        return fail(GDN_ERR_SHAPE, "without cu_seqlens num_seqs must equal batch (%d != %d)", d.num_seqs, d.batch);
    if (need && !workspace) return fail(GDN_ERR_WORKSPACE, "workspace is NULL");
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

size_t cache_dtype_size(int32_t d) { return d == GDN_E4M3 ? 1 : dtype_size(d); }

gdn_status check_cache_desc(const gdn_cache_desc *d, int32_t num_seqs) {
    if (!d) return fail(GDN_ERR_NULL, "desc is NULL");
    if (!valid_dtype(d->dtype) && d->dtype != GDN_E4M3) return fail(GDN_ERR_DTYPE, "unknown dtype code %d", d->dtype);
    if (d->slots < 1 || d->kv_heads < 1 || d->window < 1 || d->sinks < 0 || num_seqs < 0)
        return fail(GDN_ERR_SHAPE, "need slots >= 1, kv_heads >= 1, window >= 1, sinks >= 0, num_seqs >= 0 (got %d, %d, "
                    "%d, %d, %d)", d->slots, d->kv_heads, d->window, d->sinks, num_seqs);
    if (d->slots > kCacheMaxSlots || d->kv_heads > 1024 || num_seqs > kCacheMaxSeqs)
        return fail(GDN_ERR_UNSUPPORTED, "slots %d, kv_heads %d, num_seqs %d not built (at most %d, 1024, %d)", d->slots,
                    d->kv_heads, num_seqs, kCacheMaxSlots, kCacheMaxSeqs);
    if (!(d->dim == 32 || d->dim == 64 || d->dim == 128 || d->dim == 256))
        return fail(GDN_ERR_UNSUPPORTED, "dim %d not built (32, 64, 128, 256)", d->dim);
    if (d->sinks > kSwaMaxSinks)
        return fail(GDN_ERR_UNSUPPORTED, "sinks %d not built (at most %d)", d->sinks, kSwaMaxSinks);
    if ((int64_t)d->window + d->sinks >= (1 << 28)) return fail(GDN_ERR_UNSUPPORTED, "sinks + window too large");
    return GDN_OK;
}

// Type of a call's tensors: the cache's own, or any beside 8 bits.
gdn_status check_cache_type(const gdn_cache_desc &d, int32_t dtype) {
    if (!valid_dtype(dtype)) return fail(GDN_ERR_DTYPE, "unknown dtype code %d", dtype);
    if (d.dtype != GDN_E4M3 && dtype != d.dtype)
        return fail(GDN_ERR_UNSUPPORTED, "dtype %d on a cache of dtype %d not built", dtype, d.dtype);
    return GDN_OK;
}

gdn_status check_cache_seqs(const gdn_cache_desc &d, int32_t num_seqs, const int32_t *slots, const float *scales) {
    if (!slots && num_seqs > d.slots)
        return fail(GDN_ERR_SHAPE, "%d sequences on %d slots need slots", num_seqs, d.slots);
    if (!scales != (d.dtype != GDN_E4M3))
        return fail(d.dtype == GDN_E4M3 ? GDN_ERR_NULL : GDN_ERR_UNSUPPORTED, "scales go with an E4M3 cache alone");
    return GDN_OK;
}

CacheArgs cache_args(const gdn_cache_desc &d, int32_t num_seqs, int32_t tokens, int32_t dtype) {
    CacheArgs a{};
    a.P = d.slots, a.KV = d.kv_heads, a.window = d.window, a.sinks = d.sinks, a.D = d.dim, a.cache_dtype = d.dtype;
    a.N = num_seqs, a.tokens = tokens, a.dtype = dtype;
    return a;
}

size_t cache_rows(const gdn_cache_desc &d) { return 2 * (size_t)d.slots * d.kv_heads * ((size_t)d.window + d.sinks); }

// gdn_cache_write and gdn_cache_read: the same checks, another direction.
gdn_status cache_call(const gdn_cache_desc *desc, int32_t num_seqs, int32_t tokens, int32_t dtype, const void *k,
                      const void *v, const int32_t *cu_seqlens, const int32_t *lengths, const int32_t *slots,
                      const void *cache, const float *scales, int32_t *status, bool read, hipStream_t stream) {
    gdn_status s = check_cache_desc(desc, num_seqs);
    if (s != GDN_OK) return s;
    const gdn_cache_desc &d = *desc;
    s = check_cache_type(d, dtype);
    if (s != GDN_OK) return s;
    if (tokens < 0 || tokens >= (1 << 30)) return fail(GDN_ERR_SHAPE, "tokens %d out of range", tokens);
    if (!cu_seqlens && (num_seqs ? tokens % num_seqs : tokens))
        return fail(GDN_ERR_SHAPE, "without cu_seqlens tokens %d must be a multiple of num_seqs %d", tokens, num_seqs);
    s = check_cache_seqs(d, num_seqs, slots, scales);
    if (s != GDN_OK) return s;
    const size_t moved = (size_t)tokens * d.kv_heads * d.dim * dtype_size(dtype), idx = 4 * (size_t)num_seqs;
    const size_t rows = cache_rows(d);
    const bool some = num_seqs > 0;
    const Arg args[] = {{"k", k, moved, some && tokens > 0, read, 16},
                        {"v", v, moved, some && tokens > 0, read, 16},
                        {"cu_seqlens", cu_seqlens, idx + 4, false, false, 4},
                        {"lengths", lengths, idx, some && read, false, 4},
                        {"slots", slots, idx, false, false, 4},
                        {"cache", cache, rows * d.dim * cache_dtype_size(d.dtype), some, !read, 16},
                        {"scales", scales, rows * 4, false, !read, 4},
                        {"status", status, 8, false, true, 4}};
    s = check_args(args, 8);
    if (s == GDN_OK) s = check_overlap(args, 8);
    if (s != GDN_OK) return s;
    if (!some && !status) return ok();
    CacheArgs a = cache_args(d, num_seqs, tokens, dtype);
    a.cache = const_cast<void *>(cache), a.scales = const_cast<float *>(scales);
    a.lengths = lengths, a.slots = slots, a.cu = cu_seqlens, a.k = k, a.v = v, a.status = status;
    hipError_t err = read ? launch_cache_read(a, stream) : launch_cache_write(a, stream);
    if (err != hipSuccess) return hip_fail(err, read ? "gdn_cache_read launch" : "gdn_cache_write launch");
    return ok();
}

gdn_status check_step(const gdn_cache_desc *desc, int32_t num_seqs, int32_t heads) {
    gdn_status s = check_cache_desc(desc, num_seqs);
    return s == GDN_OK ? check_heads(heads, desc->kv_heads) : s;
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
    const size_t need = cu_seqlens ? swa_workspace_layout(a, false).total : 0;
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
                        {"workspace", workspace, need, false, true, 16}};
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

gdn_status gdn_cache_write(const gdn_cache_desc *desc, int32_t num_seqs, int32_t tokens, int32_t in_dtype,
                           const void *k, const void *v, const int32_t *cu_seqlens, const int32_t *lengths,
                           const int32_t *slots, void *cache, float *scales, int32_t *status, hipStream_t stream) {
    return cache_call(desc, num_seqs, tokens, in_dtype, k, v, cu_seqlens, lengths, slots, cache, scales, status, false,
                      stream);
}

gdn_status gdn_cache_read(const gdn_cache_desc *desc, int32_t num_seqs, int32_t tokens, int32_t out_dtype,
                          const void *cache, const float *scales, const int32_t *lengths, const int32_t *slots,
                          const int32_t *cu_seqlens, void *k, void *v, int32_t *status, hipStream_t stream) {
    return cache_call(desc, num_seqs, tokens, out_dtype, k, v, cu_seqlens, lengths, slots, cache, scales, status, true,
                      stream);
}

gdn_status gdn_swa_step_workspace_size(const gdn_cache_desc *desc, int32_t num_seqs, int32_t heads, size_t *bytes) {
    if (!bytes) return fail(GDN_ERR_NULL, "bytes is NULL");
    gdn_status s = check_step(desc, num_seqs, heads);
    if (s != GDN_OK) return s;
    SwaStepArgs a{};
    a.c = cache_args(*desc, num_seqs, num_seqs, GDN_FP32);
    a.H = heads;
    *bytes = swa_step_workspace(a);
    return ok();
}

gdn_status gdn_swa_step(const gdn_cache_desc *desc, int32_t num_seqs, int32_t heads, int32_t dtype, float scale,
                        const void *q, const void *k, const void *v, const int32_t *lengths, const int32_t *slots,
                        void *cache, float *scales, void *o, void *workspace, size_t workspace_bytes,
                        int32_t *status, hipStream_t stream) {
    gdn_status s = check_step(desc, num_seqs, heads);
    if (s != GDN_OK) return s;
    const gdn_cache_desc &d = *desc;
    s = check_cache_type(d, dtype);
    if (s != GDN_OK) return s;
    if (dtype == GDN_FP32 && d.dim > 128) return fail(GDN_ERR_UNSUPPORTED, "dim %d not built with FP32", d.dim);
    s = check_scale(scale);
    if (s != GDN_OK) return s;
    s = check_cache_seqs(d, num_seqs, slots, scales);
    if (s != GDN_OK) return s;
    SwaStepArgs a{};
    a.c = cache_args(d, num_seqs, num_seqs, dtype);
    a.H = heads, a.scale = scale;
    const size_t need = swa_step_workspace(a);
    if (need && !workspace) return fail(GDN_ERR_WORKSPACE, "workspace is NULL");
    if (need && workspace_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace has %zu bytes, this call needs %zu", workspace_bytes, need);
    const size_t row = (size_t)d.dim * dtype_size(dtype), idx = 4 * (size_t)num_seqs, rows = cache_rows(d);
    const bool some = num_seqs > 0;
    const Arg args[] = {{"q", q, (size_t)num_seqs * heads * row, some, false, 16},
                        {"k", k, (size_t)num_seqs * d.kv_heads * row, some, false, 16},
                        {"v", v, (size_t)num_seqs * d.kv_heads * row, some, false, 16},
                        {"lengths", lengths, idx, some, false, 4},
                        {"slots", slots, idx, false, false, 4},
                        {"cache", cache, rows * d.dim * cache_dtype_size(d.dtype), some, true, 16},
                        {"scales", scales, rows * 4, false, true, 4},
                        {"o", o, (size_t)num_seqs * heads * row, some, true, 16},
                        {"workspace", workspace, need, false, true, 16},
                        {"status", status, 8, false, true, 4}};
    s = check_args(args, 10);
    if (s == GDN_OK) s = check_overlap(args, 10);
    if (s != GDN_OK) return s;
    if (!some && !status) return ok();
    a.c.cache = cache, a.c.scales = scales, a.c.lengths = lengths, a.c.slots = slots, a.c.k = k, a.c.v = v;
    a.c.status = status;
    a.q = q, a.o = o, a.workspace = workspace;
    hipError_t err = launch_swa_step(a, stream);
    if (err != hipSuccess) return hip_fail(err, "gdn_swa_step launch");
    return ok();
}

}  // extern "C"
