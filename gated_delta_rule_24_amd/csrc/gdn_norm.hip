// Layer norm and its gradient (HBM-bound).
#include "gdn_device.h"
#include "gdn_ops.h"
#include "gdn_types.h"

namespace gdn {

// Sum over a 256-thread block; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float *s) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// One block per row.
template <typename x_t, typename y_t>
__global__ __launch_bounds__(256) void layernorm_fwd_kernel(int D, float eps, const x_t *__restrict__ x,
                                                            const float *__restrict__ w, const float *__restrict__ b,
                                                            y_t *__restrict__ y, float *__restrict__ mean,
                                                            float *__restrict__ rstd) {
    __shared__ float s[4];
    const int64_t r = blockIdx.x;
    const x_t *row = x + r * D;
    float m = 0.f, v = 0.f;
    for (int i = threadIdx.x; i < D; i += 256) m += to_f32(row[i]);
    m = block_sum(m, s) / D;
    for (int i = threadIdx.x; i < D; i += 256) {
        const float c = to_f32(row[i]) - m;
        v += c * c;
    }
    const float q = 1.f / sqrtf(block_sum(v, s) / D + eps);
    for (int i = threadIdx.x; i < D; i += 256)
        y[r * D + i] = round_to<y_t>((to_f32(row[i]) - m) * q * (w ? w[i] : 1.f) + (b ? b[i] : 0.f));
    if (mean && threadIdx.x == 0) {
        mean[r] = m;
        rstd[r] = q;
    }
}

template <typename x_t, typename y_t>
__global__ __launch_bounds__(256) void layernorm_dx_kernel(int D, const y_t *__restrict__ dy,
                                                           const x_t *__restrict__ x, const float *__restrict__ mean,
                                                           const float *__restrict__ rstd,
                                                           const float *__restrict__ w, x_t *__restrict__ dx) {
    __shared__ float s[4];
    const int64_t r = blockIdx.x;
    const float m = mean[r], q = rstd[r];
    float c1 = 0.f, c2 = 0.f;
    for (int i = threadIdx.x; i < D; i += 256) {
        const float u = to_f32(dy[r * D + i]) * (w ? w[i] : 1.f);
        c1 += u;
        c2 += u * (to_f32(x[r * D + i]) - m) * q;
    }
    c1 = block_sum(c1, s) / D;
    c2 = block_sum(c2, s) / D;
    for (int i = threadIdx.x; i < D; i += 256) {
        const float u = to_f32(dy[r * D + i]) * (w ? w[i] : 1.f);
        dx[r * D + i] = round_to<x_t>(q * (u - c1 - (to_f32(x[r * D + i]) - m) * q * c2));
    }
}

// One thread per column and one of 16 row groups; the groups join in LDS.
template <typename x_t, typename y_t>
__global__ __launch_bounds__(1024) void layernorm_dw_kernel(int64_t rows, int D, const y_t *__restrict__ dy,
                                                            const x_t *__restrict__ x,
                                                            const float *__restrict__ mean,
                                                            const float *__restrict__ rstd, float *__restrict__ dw,
                                                            float *__restrict__ db) {
    __shared__ float sw[16][64], sb[16][64];
    const int c = threadIdx.x & 63, g = threadIdx.x >> 6, d = blockIdx.x * 64 + c;
    float aw = 0.f, ab = 0.f;
    if (d < D)
        for (int64_t r = g; r < rows; r += 16) {
            const float v = to_f32(dy[r * D + d]);
            aw += v * (to_f32(x[r * D + d]) - mean[r]) * rstd[r];
            ab += v;
        }
    sw[g][c] = aw;
    sb[g][c] = ab;
    __syncthreads();
    if (g == 0 && d < D) {
        for (int i = 1; i < 16; ++i) {
            aw += sw[i][c];
            ab += sb[i][c];
        }
        if (dw) dw[d] = aw;
        if (db) db[d] = ab;
    }
}

size_t layernorm_bwd_workspace(int64_t, int32_t) { return 256; }

hipError_t launch_layernorm_fwd(const NormArgs &a, hipStream_t st) {
    ProfScope prof("gdn_layernorm_fwd", st);
    return with_types(a.in_dtype, a.out_dtype, a.in_dtype, [&](auto x, auto y, auto) {
        using x_t = decltype(x);
        using y_t = decltype(y);
        layernorm_fwd_kernel<x_t, y_t><<<(unsigned)a.rows, 256, 0, st>>>(
            a.dim, a.eps, static_cast<const x_t *>(a.x), a.weight, a.bias, static_cast<y_t *>(a.y), a.mean, a.rstd);
        return hipGetLastError();
    });
}

hipError_t launch_layernorm_bwd(const NormArgs &a, hipStream_t st) {
    ProfScope prof("gdn_layernorm_bwd", st);
    return with_types(a.in_dtype, a.out_dtype, a.in_dtype, [&](auto x, auto y, auto) {
        using x_t = decltype(x);
        using y_t = decltype(y);
        auto *dy = static_cast<const y_t *>(a.dy);
        auto *xx = static_cast<const x_t *>(a.x);
        if (a.rows)
            layernorm_dx_kernel<x_t, y_t><<<(unsigned)a.rows, 256, 0, st>>>(a.dim, dy, xx, a.mean, a.rstd, a.weight,
                                                                            static_cast<x_t *>(a.dx));
        if (a.dweight || a.dbias)
            layernorm_dw_kernel<x_t, y_t><<<(unsigned)((a.dim + 63) / 64), 1024, 0, st>>>(
                a.rows, a.dim, dy, xx, a.mean, a.rstd, a.dweight, a.dbias);
        return hipGetLastError();
    });
}

}  // namespace gdn
