// Gated linear recurrence h_t = alpha_t h_{t-1} + x_t per channel, its
// gradient and its single step (HBM-bound: no value is used twice).
#include "gdn_device.h"
#include "gdn_ops.h"
#include "gdn_types.h"

namespace gdn {

ScanWorkspace scan_workspace_layout(int32_t, int32_t, int32_t, int32_t N, bool packed) {
    ScanWorkspace w;
    w.off_meta = 0;
    w.off_cu = 256;
    w.total = 256 + (packed ? ((size_t)(N + 1) * 4 + 255) / 256 * 256 : 0);
    return w;
}

// One thread per (sequence, channel), token by token.
template <typename x_t, typename l_t, typename h_t>
__global__ __launch_bounds__(64) void scan_fwd_kernel(int T, int D, const int32_t *__restrict__ cu,
                                                       const int32_t *__restrict__ meta, const x_t *__restrict__ x,
                                                       const l_t *__restrict__ la, const float *init,
                                                       float *final_state, h_t *__restrict__ h) {
    if (cu && meta[1] != 0) return;
    const int n = blockIdx.x, d = blockIdx.y * 64 + threadIdx.x;
    if (d >= D) return;
    const int64_t t0 = cu ? cu[n] : (int64_t)n * T, t1 = cu ? cu[n + 1] : t0 + T;
    float s = init ? init[(int64_t)n * D + d] : 0.f;
    for (int64_t t = t0; t < t1; ++t) {
        s = expf(to_f32(la[t * D + d])) * s + to_f32(x[t * D + d]);
        h[t * D + d] = round_to<h_t>(s);
    }
    if (final_state) final_state[(int64_t)n * D + d] = s;
}

template <typename x_t, typename l_t, typename h_t>
__global__ __launch_bounds__(64) void scan_bwd_kernel(int T, int D, const int32_t *__restrict__ cu,
                                                       const int32_t *__restrict__ meta, const l_t *__restrict__ la,
                                                       const h_t *__restrict__ h, const float *__restrict__ init,
                                                       const h_t *__restrict__ dh, const float *__restrict__ dfin,
                                                       x_t *__restrict__ dx, l_t *__restrict__ dla,
                                                       float *__restrict__ dinit) {
    if (cu && meta[1] != 0) return;
    const int n = blockIdx.x, d = blockIdx.y * 64 + threadIdx.x;
    if (d >= D) return;
    const int64_t t0 = cu ? cu[n] : (int64_t)n * T, t1 = cu ? cu[n + 1] : t0 + T;
    float e = dfin ? dfin[(int64_t)n * D + d] : 0.f;
    for (int64_t t = t1 - 1; t >= t0; --t) {
        const float g = to_f32(dh[t * D + d]) + e;
        e = expf(to_f32(la[t * D + d])) * g;
        const float before = t > t0 ? to_f32(h[(t - 1) * D + d]) : (init ? init[(int64_t)n * D + d] : 0.f);
        dx[t * D + d] = round_to<x_t>(g);
        dla[t * D + d] = round_to<l_t>(e * before);
    }
    if (dinit) dinit[(int64_t)n * D + d] = e;
}

static hipError_t check_cu(const ScanArgs &a, hipStream_t st) {
    if (!a.cu_seqlens) return hipSuccess;
    const auto w = scan_workspace_layout(a.B, a.T, a.D, a.N, true);
    char *ws = static_cast<char *>(a.workspace);
    return launch_chunk_table(a.N, a.T, a.cu_seqlens, reinterpret_cast<int32_t *>(ws + w.off_meta),
                              reinterpret_cast<int32_t *>(ws + w.off_cu), nullptr, nullptr, nullptr, 0, nullptr,
                              nullptr, nullptr, st, false);
}

hipError_t launch_scan_fwd(const ScanArgs &a, hipStream_t st) {
    hipError_t e = check_cu(a, st);
    if (e != hipSuccess) return e;
    ProfScope prof("gdn_scan_fwd", st);
    return with_types(a.in_dtype, a.gate_dtype, a.out_dtype, [&](auto x, auto l, auto h) {
        using x_t = decltype(x);
        using l_t = decltype(l);
        using h_t = decltype(h);
        scan_fwd_kernel<x_t, l_t, h_t><<<dim3(a.N, (a.D + 63) / 64), 64, 0, st>>>(
            a.T, a.D, a.cu_seqlens, static_cast<const int32_t *>(a.workspace), static_cast<const x_t *>(a.x),
            static_cast<const l_t *>(a.log_alpha), a.init_state, a.final_state, static_cast<h_t *>(a.h));
        return hipGetLastError();
    });
}

hipError_t launch_scan_bwd(const ScanArgs &a, hipStream_t st) {
    hipError_t e = check_cu(a, st);
    if (e != hipSuccess) return e;
    ProfScope prof("gdn_scan_bwd", st);
    return with_types(a.in_dtype, a.gate_dtype, a.out_dtype, [&](auto x, auto l, auto h) {
        using x_t = decltype(x);
        using l_t = decltype(l);
        using h_t = decltype(h);
        scan_bwd_kernel<x_t, l_t, h_t><<<dim3(a.N, (a.D + 63) / 64), 64, 0, st>>>(
            a.T, a.D, a.cu_seqlens, static_cast<const int32_t *>(a.workspace), static_cast<const l_t *>(a.log_alpha),
            static_cast<const h_t *>(a.h), a.init_state, static_cast<const h_t *>(a.d_h), a.d_final,
            static_cast<x_t *>(a.dx), static_cast<l_t *>(a.dlog_alpha), a.d_init);
        return hipGetLastError();
    });
}

template <typename x_t, typename l_t, typename h_t>
__global__ __launch_bounds__(256) void scan_step_kernel(int64_t n, float *__restrict__ state,
                                                        const x_t *__restrict__ x, const l_t *__restrict__ la,
                                                        h_t *__restrict__ h) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const float s = expf(to_f32(la[i])) * state[i] + to_f32(x[i]);
        state[i] = s;
        h[i] = round_to<h_t>(s);
    }
}

hipError_t launch_scan_step(const ScanStepArgs &a, hipStream_t st) {
    const int64_t n = (int64_t)a.N * a.D;
    const int64_t blocks = (n + 255) / 256;
    ProfScope prof("gdn_scan_step", st);
    return with_types(a.in_dtype, a.gate_dtype, a.out_dtype, [&](auto x, auto l, auto h) {
        using x_t = decltype(x);
        using l_t = decltype(l);
        using h_t = decltype(h);
        scan_step_kernel<x_t, l_t, h_t><<<(unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)), 256, 0, st>>>(
            n, a.state, static_cast<const x_t *>(a.x), static_cast<const l_t *>(a.log_alpha),
            static_cast<h_t *>(a.h));
        return hipGetLastError();
    });
}

}  // namespace gdn
