// Error reporting and argument predicates shared by the C ABI files.
#pragma once

#include "gdn.h"

#include <stddef.h>
#include <stdint.h>

namespace gdn {

// Store the thread's error message and return the status (gdn_api.cpp).
gdn_status fail(gdn_status s, const char *fmt, ...);
gdn_status ok();
gdn_status hip_fail(hipError_t e, const char *what);

inline bool valid_dtype(int32_t d) { return d == GDN_FP32 || d == GDN_BF16 || d == GDN_FP16; }
inline size_t dtype_size(int32_t d) { return d == GDN_FP32 ? 4 : 2; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Range {
    const char *name;
    uintptr_t lo, hi;   // [lo, hi)
};
inline Range rng(const char *name, const void *p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{name, lo, p ? lo + bytes : lo};
}
inline bool overlap(const Range &a, const Range &b) {
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

// A pointer argument with what is checked of it.
struct Arg {
    const char *name;
    const void *p;
    size_t bytes;
    bool required, written;
    int align;
};

inline gdn_status check_args(const Arg *a, int n) {
    for (int i = 0; i < n; ++i)
        if (a[i].required && !a[i].p) return fail(GDN_ERR_NULL, "%s is required", a[i].name);
    for (int i = 0; i < n; ++i)
        if (a[i].p && (reinterpret_cast<uintptr_t>(a[i].p) & (a[i].align - 1)))
            return fail(GDN_ERR_ALIGN, "%s is not %d-byte aligned", a[i].name, a[i].align);
    return GDN_OK;
}

// No written range may overlap another one; `same`: the one pair that may be
// the same buffer.
inline gdn_status check_overlap(const Arg *a, int n, int same0 = -1, int same1 = -1) {
    for (int i = 0; i < n; ++i) {
        if (!a[i].written) continue;
        for (int j = 0; j < n; ++j) {
            if (i == j || (a[j].written && j < i)) continue;
            if (((i == same0 && j == same1) || (i == same1 && j == same0)) && a[i].p == a[j].p) continue;
            if (overlap(rng(a[i].name, a[i].p, a[i].bytes), rng(a[j].name, a[j].p, a[j].bytes)))
                return fail(GDN_ERR_ALIAS, "%s overlaps %s", a[i].name, a[j].name);
        }
    }
    return GDN_OK;
}

// Each type fp32 or one 16-bit type.
inline gdn_status check_types(const int32_t *dt, int n) {
    int32_t half = GDN_FP32;
    for (int i = 0; i < n; ++i) {
        if (!valid_dtype(dt[i])) return fail(GDN_ERR_DTYPE, "unknown dtype code %d", dt[i]);
        if (dt[i] == GDN_FP32) continue;
        if (half != GDN_FP32 && half != dt[i])
            return fail(GDN_ERR_UNSUPPORTED, "bf16 and fp16 do not mix in one call");
        half = dt[i];
    }
    return GDN_OK;
}

}  // namespace gdn
