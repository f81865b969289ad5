// The resident cache of windowed attention: rows of its 8-bit form, which the
// kernels that write, read and attend to it share, and their arguments.
#pragma once

#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_types.h"

namespace gdn {

constexpr int32_t DT_E4M3 = 3;
constexpr int kCacheMaxSeqs = 4096, kCacheMaxSlots = 65536;
constexpr int32_t kCacheMaxLength = 1 << 30;      // positions

struct CacheArgs {
    int32_t P, KV, window, sinks, D, cache_dtype, N, tokens, dtype;
    void *cache;                    // [2, P, KV, sinks + window, D]
    float *scales;                  // [2, P, KV, sinks + window], 8 bits only
    const int32_t *lengths, *slots, *cu;
    const void *k, *v;              // write: read; read: written
    int32_t *status;
};
hipError_t launch_cache_write(const CacheArgs &a, hipStream_t stream);
hipError_t launch_cache_read(const CacheArgs &a, hipStream_t stream);

struct SwaStepArgs {
    CacheArgs c;                    // k, v: the new token's
    int32_t H;
    float scale;
    const void *q;
    void *o, *workspace;
};
// Parts of the rows, each a block's, and the workspace for their results.
int swa_step_splits(const SwaStepArgs &a);
size_t swa_step_workspace(const SwaStepArgs &a);
hipError_t launch_swa_step(const SwaStepArgs &a, hipStream_t stream);

// A slot of the call: the index is in range, or -1 (the sequence is left out).
__device__ __forceinline__ bool slot_in_range(int s, int slots) { return s >= -1 && s < slots; }

// The cache row of position p: the sinks' own, then a ring.
__device__ __forceinline__ int cache_row(int p, int window, int sinks) {
    return p < sinks ? p : sinks + (p - sinks) % window;
}

// ---- 8-bit rows ------------------------------------------------------------------
//
// e4m3 values with one power of two per row (token, head): scale = 2^e with the
// least e >= -126 for which max|x| <= 448 * 2^e.  The division is exact, so the one
// rounding is that to e4m3; reading back is exact.  A power of two loses nothing
// against max|x| / 448 but half of the smallest values' range (2^-9 of the scale),
// and needs no rounding of its own.  A row that is not finite gets the scale NaN.

__device__ __forceinline__ float e4m3_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    if (!(amax < __builtin_inff())) return __builtin_nanf("");
    const int b = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u);   // 448 = 1.75 * 2^8
    return __uint_as_float((uint32_t)(b < 1 ? 1 : b) << 23);
}
__device__ __forceinline__ float e4m3_inverse(float scale) {
    return scale == scale ? __uint_as_float((254u << 23) - __float_as_uint(scale)) : scale;
}
// Eight values, already divided, as e4m3 (round to nearest even).
__device__ __forceinline__ uint2 to_e4m3(const float (&x)[8]) {
    uint2 r;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    r.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], 0, false);
    r.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], w, true);
    return r;
}
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void from_e4m3(uint32_t w, float (&x)[4]) {
    const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
}

// Largest |x| of a row whose D elements lie eight to a lane; NaN where one is.
template <int L>
__device__ __forceinline__ float row_amax(const float (&x)[8]) {
    float m = 0.f, nan = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        m = fmaxf(m, fabsf(x[e]));
        nan = x[e] != x[e] ? 1.f : nan;
    }
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1) {
        m = fmaxf(m, __shfl_xor(m, d, 64));
        nan = fmaxf(nan, __shfl_xor(nan, d, 64));
    }
    return nan > 0.f ? __builtin_nanf("") : m;
}

}  // namespace gdn
