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

}  // namespace gdn
