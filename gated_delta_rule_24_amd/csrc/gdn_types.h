// Dispatch on the element types of a call: each of its types is fp32 or one
// 16-bit type (include/gdn.h), so a kernel with three typed tensors has 15
// instantiations.
#pragma once

#include "gdn_device.h"
#include "gdn_launch.h"

#include <type_traits>

namespace gdn {

// The fp32 value `x` rounded to T.  The empty asm keeps the compiler from
// joining the conversion to fp16 with the multiply-add that made x, which
// would round the unrounded sum instead of the fp32 value that is kept.
template <typename T>
__device__ __forceinline__ T round_to(float x) {
    if constexpr (std::is_same_v<T, _Float16>) asm("" : "+v"(x));
    return from_f32<T>(x);
}

// f(A{}, B{}, C{}) with the types that the codes name.
template <typename T, typename F>
hipError_t with_types3_of(int32_t a, int32_t b, int32_t c, F f) {
    auto third = [&](auto x, auto y) {
        return c == DT_FP32 ? f(x, y, float{}) : f(x, y, T{});
    };
    auto second = [&](auto x) {
        return b == DT_FP32 ? third(x, float{}) : third(x, T{});
    };
    return a == DT_FP32 ? second(float{}) : second(T{});
}
template <typename F>
hipError_t with_types(int32_t a, int32_t b, int32_t c, F f) {
    if (a == DT_BF16 || b == DT_BF16 || c == DT_BF16) return with_types3_of<bf16_t>(a, b, c, f);
    if (a == DT_FP16 || b == DT_FP16 || c == DT_FP16) return with_types3_of<_Float16>(a, b, c, f);
    return f(float{}, float{}, float{});
}

}  // namespace gdn
