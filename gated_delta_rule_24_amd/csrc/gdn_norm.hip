// Layer norm over rows and its gradient.  Both are bound by HBM: a row is read
// once into registers and its statistics are taken from there, the mean first
// and then the squares about it, so rows far from zero keep their variance.
//
// A row belongs to L lanes (a power of two): part of a wave for short rows,
// so that a wave takes several, or whole waves that join through LDS.  Every
// lane holds K groups of 8 elements.  Where D is a multiple of 8 a group is 8
// neighbours, loaded as one or two 16-byte vectors; otherwise rows do not
// start on a vector and a group is 8 elements L apart, so that lanes still
// load neighbours.
//
// The gradients of weight and bias are sums over rows.  A block walks over
// rows a grid apart and keeps its columns' sums in registers, its row groups
// join in LDS, and each block writes one line of partial sums; a second
// kernel adds the lines.  The order is fixed by the shape, so equal calls
// give equal bits.
#include "gdn_device.h"
#include "gdn_ops.h"
#include "gdn_types.h"

namespace gdn {

// Layout of one row over a block.
template <int L_, int K_, int NT_, bool VEC_>
struct RowShape {
    static constexpr int L = L_;         // lanes per row
    static constexpr int K = K_;         // groups of 8 elements per lane
    static constexpr int NT = NT_;       // threads of the block
    static constexpr bool VEC = VEC_;
    static constexpr int ROWS = NT / L;  // rows of a block at a time
    static constexpr int E = 8 * K;      // elements per lane
    // column of element e of group k for lane l
    __device__ __forceinline__ static int col(int l, int k, int e) {
        return VEC ? (k * L + l) * 8 + e : (k * 8 + e) * L + l;
    }
};

// Elements of a row that lane l holds, as fp32; 0 past the row's end.
template <typename S, typename T>
__device__ __forceinline__ void load_row(const T *__restrict__ row, int D, int l, float (&v)[S::E]) {
#pragma unroll
    for (int k = 0; k < S::K; ++k) {
        if constexpr (S::VEC) {
            const int c = S::col(l, k, 0);
            float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (c < D) load8_f32(row + c, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * k + e] = o[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = S::col(l, k, e);
                v[8 * k + e] = c < D ? to_f32(row[c]) : 0.f;
            }
        }
    }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    if constexpr (std::is_same_v<T, float>) {
        reinterpret_cast<float4_t *>(p)[0] = float4_t{v[0], v[1], v[2], v[3]};
        reinterpret_cast<float4_t *>(p)[1] = float4_t{v[4], v[5], v[6], v[7]};
    } else {
        struct alignas(16) O {
            T e[8];
        } o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.e[e] = round_to<T>(v[e]);
        *reinterpret_cast<O *>(p) = o;
    }
}
template <typename S, typename T>
__device__ __forceinline__ void store_row(T *__restrict__ row, int D, int l, const float (&v)[S::E]) {
#pragma unroll
    for (int k = 0; k < S::K; ++k) {
        if constexpr (S::VEC) {
            const int c = S::col(l, k, 0);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = v[8 * k + e];
            if (c < D) store8(row + c, o);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = S::col(l, k, e);
                if (c < D) row[c] = round_to<T>(v[8 * k + e]);
            }
        }
    }
}

// Sums of two values over the lanes of a row (L lanes; whole waves join in
// LDS, each row of the block in its own words).  Every lane gets the sums.
template <typename S>
__device__ __forceinline__ void row_sum2(float &a, float &b, float (*s)[2]) {
    constexpr int W = S::L < 64 ? S::L : 64;
#pragma unroll
    for (int m = W / 2; m >= 1; m >>= 1) {
        a += __shfl_xor(a, m, 64);
        b += __shfl_xor(b, m, 64);
    }
    if constexpr (S::L > 64) {
        constexpr int NW = S::L / 64;
        const int w = threadIdx.x / 64, w0 = w / NW * NW;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) s[w][0] = a, s[w][1] = b;
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) a += s[w0 + i][0], b += s[w0 + i][1];
    }
}

template <typename S, typename x_t, typename y_t>
__global__ __launch_bounds__(S::NT) void layernorm_fwd_kernel(int64_t rows, int D, float eps,
                                                              const x_t *__restrict__ x, const float *__restrict__ w,
                                                              const float *__restrict__ b, y_t *__restrict__ y,
                                                              float *__restrict__ mean, float *__restrict__ rstd) {
    __shared__ float s[S::NT / 64][2];
    const int l = threadIdx.x % S::L, g = threadIdx.x / S::L;
    float wv[S::E], bv[S::E];
    if (w) load_row<S>(w, D, l, wv);
    if (b) load_row<S>(b, D, l, bv);
    const float n = (float)D;
    for (int64_t r0 = (int64_t)blockIdx.x * S::ROWS; r0 < rows; r0 += (int64_t)gridDim.x * S::ROWS) {
        const int64_t r = r0 + g;
        const bool on = r < rows;
        float v[S::E];
        load_row<S>(x + (on ? r : 0) * D, D, l, v);
        float m = 0.f, q = 0.f, none = 0.f;
#pragma unroll
        for (int e = 0; e < S::E; ++e) m += v[e];
        row_sum2<S>(m, none, s);
        m /= n;
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float &c = v[8 * k + e];
                c = S::col(l, k, S::VEC ? 0 : e) < D ? c - m : 0.f;
                q = fmaf(c, c, q);
            }
        row_sum2<S>(q, none, s);
        q = 1.f / sqrtf(q / n + eps);
#pragma unroll
        for (int e = 0; e < S::E; ++e) {
            v[e] *= q;
            if (w) v[e] *= wv[e];
            if (b) v[e] += bv[e];
        }
        if (on) {
            store_row<S>(y + r * D, D, l, v);
            if (mean && l == 0) {
                mean[r] = m;
                rstd[r] = q;
            }
        }
    }
}

// SUMS: also the block's line of partial sums, part[block][2][D].
template <typename S, typename x_t, typename y_t, bool SUMS>
__global__ __launch_bounds__(S::NT) void layernorm_bwd_kernel(int64_t rows, int D, const y_t *__restrict__ dy,
                                                              const x_t *__restrict__ x,
                                                              const float *__restrict__ mean,
                                                              const float *__restrict__ rstd,
                                                              const float *__restrict__ w, x_t *__restrict__ dx,
                                                              float *__restrict__ part) {
    __shared__ float s[S::NT / 64][2];
    const int l = threadIdx.x % S::L, g = threadIdx.x / S::L;
    float wv[S::E], aw[S::E], ab[S::E];
    if (w) load_row<S>(w, D, l, wv);
#pragma unroll
    for (int e = 0; e < S::E; ++e) aw[e] = ab[e] = 0.f;
    const float n = (float)D;
    for (int64_t r0 = (int64_t)blockIdx.x * S::ROWS; r0 < rows; r0 += (int64_t)gridDim.x * S::ROWS) {
        const int64_t r = r0 + g;
        const bool on = r < rows;
        const int64_t rr = on ? r : 0;
        float u[S::E], c[S::E];
        load_row<S>(dy + rr * D, D, l, u);
        load_row<S>(x + rr * D, D, l, c);
        const float m = mean[rr], q = rstd[rr];
        float c1 = 0.f, c2 = 0.f;
#pragma unroll
        for (int e = 0; e < S::E; ++e) {
            c[e] = (c[e] - m) * q;                  // past the row's end u = 0, so c counts for nothing there
            if (SUMS && on) {
                aw[e] = fmaf(u[e], c[e], aw[e]);
                ab[e] += u[e];
            }
            if (w) u[e] *= wv[e];
            c1 += u[e];
            c2 = fmaf(u[e], c[e], c2);
        }
        row_sum2<S>(c1, c2, s);
        c1 /= n;
        c2 /= n;
#pragma unroll
        for (int e = 0; e < S::E; ++e) u[e] = q * (u[e] - c1 - c[e] * c2);
        if (on) store_row<S>(dx + r * D, D, l, u);
    }
    if constexpr (SUMS) {
        // the block's row groups join, a part of the columns at a time
        float *line = part + (int64_t)blockIdx.x * 2 * D;
        if constexpr (S::ROWS == 1) {
#pragma unroll
            for (int k = 0; k < S::K; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int col = S::col(l, k, e);
                    if (col < D) line[col] = aw[8 * k + e], line[D + col] = ab[8 * k + e];
                }
        } else {
            __shared__ float sw[S::NT][9], sb[S::NT][9];
#pragma unroll
            for (int k = 0; k < S::K; ++k) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 8; ++e) sw[threadIdx.x][e] = aw[8 * k + e], sb[threadIdx.x][e] = ab[8 * k + e];
                __syncthreads();
                for (int i = threadIdx.x; i < S::L * 8; i += S::NT) {
                    const int il = i >> 3, e = i & 7, col = S::col(il, k, e);
                    if (col >= D) continue;
                    float tw = 0.f, tb = 0.f;
#pragma unroll 8
                    for (int q = 0; q < S::ROWS; ++q) tw += sw[q * S::L + il][e], tb += sb[q * S::L + il][e];
                    line[col] = tw;
                    line[D + col] = tb;
                }
            }
        }
    }
}

// Adds the lines: 16 columns of the 2 D (weight's, then bias's) by 16 lanes,
// 64 groups of lines that join in LDS.
__global__ __launch_bounds__(1024) void layernorm_sums_kernel(int lines, int D, const float *__restrict__ part,
                                                              float *__restrict__ dw, float *__restrict__ db) {
    __shared__ float s[64][17];
    const int c = threadIdx.x & 15, g = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
    float a = 0.f;
    if (col < 2 * D)
#pragma unroll 4
        for (int i = g; i < lines; i += 64) a += part[(int64_t)i * 2 * D + col];
    s[g][c] = a;
    __syncthreads();
    for (int n = 32; n >= 1; n >>= 1) {
        if (g < n) s[g][c] += s[g + n][c];
        __syncthreads();
    }
    if (g == 0 && col < 2 * D) {
        if (col < D) {
            if (dw) dw[col] = s[0][c];
        } else if (db) {
            db[col - D] = s[0][c];
        }
    }
}

// f(RowShape{}) with the layout for D: as many lanes as 8 elements each need,
// up to a wave; longer rows take 16 elements a lane, then more waves.
template <bool VEC, typename F>
static hipError_t with_row_shape_of(int D, F f) {
    if (D <= 64) return f(RowShape<8, 1, 256, VEC>{});
    if (D <= 128) return f(RowShape<16, 1, 256, VEC>{});
    if (D <= 256) return f(RowShape<32, 1, 256, VEC>{});
    if (D <= 512) return f(RowShape<64, 1, 256, VEC>{});
    if (D <= 1024) return f(RowShape<64, 2, 256, VEC>{});
    if (D <= 2048) return f(RowShape<128, 2, 256, VEC>{});
    if (D <= 4096) return f(RowShape<256, 2, 256, VEC>{});
    if (D <= 8192) return f(RowShape<512, 2, 512, VEC>{});
    return f(RowShape<1024, 2, 1024, VEC>{});
}
template <typename F>
static hipError_t with_row_shape(int D, F f) {
    return D % 8 == 0 ? with_row_shape_of<true>(D, f) : with_row_shape_of<false>(D, f);
}

// Blocks of the backward kernel, and so lines of partial sums.
static int64_t bwd_blocks(int64_t rows, int rows_per_block, int threads) {
    const int64_t most = 256 * (1024 / threads);      // about 1024 threads on each of 256 CUs
    const int64_t need = (rows + rows_per_block - 1) / rows_per_block;
    return need < most ? need : most;
}

size_t layernorm_bwd_workspace(int64_t rows, int32_t dim) {
    int64_t lines = 0;
    with_row_shape(dim, [&](auto s) {
        using S = decltype(s);
        lines = bwd_blocks(rows, S::ROWS, S::NT);
        return hipSuccess;
    });
    return (size_t)(lines * 2 * dim * 4 + 255) / 256 * 256 + 256;
}

hipError_t launch_layernorm_fwd(const NormArgs &a, hipStream_t st) {
    ProfScope prof("gdn_layernorm_fwd", st);
    return with_types(a.in_dtype, a.out_dtype, a.in_dtype, [&](auto x, auto y, auto) {
        using x_t = decltype(x);
        using y_t = decltype(y);
        return with_row_shape(a.dim, [&](auto s) {
            using S = decltype(s);
            const int64_t need = (a.rows + S::ROWS - 1) / S::ROWS;
            const unsigned blocks = (unsigned)(need < (1 << 20) ? need : (1 << 20));
            layernorm_fwd_kernel<S, x_t, y_t><<<blocks, S::NT, 0, st>>>(
                a.rows, a.dim, a.eps, static_cast<const x_t *>(a.x), a.weight, a.bias, static_cast<y_t *>(a.y),
                a.mean, a.rstd);
            return hipGetLastError();
        });
    });
}

hipError_t launch_layernorm_bwd(const NormArgs &a, hipStream_t st) {
    const bool sums = a.dweight || a.dbias;
    float *part = static_cast<float *>(a.workspace);
    int64_t blocks = 0;
    hipError_t e = hipSuccess;
    if (a.rows) {
        ProfScope prof("gdn_layernorm_bwd", st);
        e = with_types(a.in_dtype, a.out_dtype, a.in_dtype, [&](auto x, auto y, auto) {
            using x_t = decltype(x);
            using y_t = decltype(y);
            return with_row_shape(a.dim, [&](auto s) {
                using S = decltype(s);
                blocks = bwd_blocks(a.rows, S::ROWS, S::NT);
                auto go = [&](auto *kernel) {
                    kernel<<<(unsigned)blocks, S::NT, 0, st>>>(
                        a.rows, a.dim, static_cast<const y_t *>(a.dy), static_cast<const x_t *>(a.x), a.mean, a.rstd,
                        a.weight, static_cast<x_t *>(a.dx), part);
                    return hipGetLastError();
                };
                return sums ? go(layernorm_bwd_kernel<S, x_t, y_t, true>)
                            : go(layernorm_bwd_kernel<S, x_t, y_t, false>);
            });
        });
    }
    if (e != hipSuccess || !sums) return e;
    ProfScope prof("gdn_layernorm_sums", st);
    layernorm_sums_kernel<<<(unsigned)((2 * a.dim + 15) / 16), 1024, 0, st>>>((int)blocks, a.dim, part, a.dweight,
                                                                            a.dbias);
    return hipGetLastError();
}

}  // namespace gdn
