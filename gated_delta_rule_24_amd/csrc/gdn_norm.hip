// Layer norm over rows and its gradient.  Both are bound by HBM: a row is read
// once into registers and its statistics are taken from there, the mean first
// and then the squares about it, so rows far from zero keep their variance.
//
// A row belongs to L lanes (a power of two): part of a wave for short rows,
// so that a wave takes several, or whole waves that join through LDS.  Every
// lane holds K groups of 8 neighbouring elements, loaded as one or two 16-byte
// vectors.  Where D is no multiple of 8 the vectors are not aligned (the
// hardware takes them as they are) and the row's last group starts earlier, so
// that it ends with the row: the elements that it shares with the group before
// count once and are written twice, with the same bits.  Rows of less than 8
// elements go one by one.  A block walks over rows a grid apart and has the
// loads of its next rows in flight while it works on a row.  The gradient of
// rows wider than 8192 does not fit: 1024 threads have 128 registers each, and up
// to 36 of what a thread holds go to scratch where D is a multiple of 8, 89 to 145
// where it is not.
//
// Measured (MI355X, a large copy reaches 5.4 TB/s): 262144 x 128 from fp32 to
// bf16 36 us (5.6 TB/s), its gradient in bf16 40 us (5.1), 16384 x 2048 in
// bf16 24 us (5.6), its gradient 43 us (4.7).  The gradient of 4093 x 1001 in fp16
// takes 17 us, 13 of them in the kernel over the rows: 128 blocks on 256 CUs, each
// with four turns behind one another and a join of its sums, then a second launch.
// Lanes per row are a power of two with one to three groups each, so widths just
// above a step leave up to half of the lanes idle; and the partial sums are
// written and read again (256 lines of 2 D: a sixth of the rows' own bytes at
// 2048 x 16384).  2^25 elements in bf16, forward and gradient in us, a copy of the
// bytes 25 and 37:
//     33  38   50       1032  27   64       4100  44   70       8200  47   67
//    264  26   52       2048  23   43       5000  26   68      12288  39   66
//    300  38   48       2050  50   61       8192  28   55      16383  50  111
//   1001  31   42       4096  24   53                          16384  40   69
//
// The gradients of weight and bias are sums over rows.  A block walks over
// rows a grid apart and keeps its columns' sums in registers, its row groups
// join in LDS, and each block writes one line of partial sums; a second
// kernel adds the lines.  The order is fixed by the shape, so equal calls
// give equal bits.
#include "gdn_device.h"
#include "gdn_ops.h"
#include "gdn_types.h"

#include <algorithm>

namespace gdn {

// Layout of one row over a block.
template <int L_, int K_, int NT_, bool WHOLE_>
struct RowShape {
    static constexpr int L = L_;         // lanes per row
    static constexpr int K = K_;         // groups of 8 elements per lane
    static constexpr int NT = NT_;       // threads of the block
    static constexpr bool WHOLE = WHOLE_;   // D is a multiple of 8
    static constexpr int ROWS = NT / L;  // rows of a block at a time
    static constexpr int E = 8 * K;      // elements per lane
    // first column of group k of lane l, and where it is loaded from
    __device__ __forceinline__ static int col(int l, int k) { return (k * L + l) * 8; }
    __device__ __forceinline__ static int from(int l, int k, int D) {
        return WHOLE ? col(l, k) : max(min(col(l, k), D - 8), 0);
    }
    // whether element e of the group, at column from() + e, counts for this lane
    __device__ __forceinline__ static bool counts(int l, int k, int e, int D) {
        const int c = col(l, k);
        return WHOLE ? c < D : c < D && from(l, k, D) + e >= c && e < D;
    }
};

typedef u32x4_t loose4_t __attribute__((aligned(2)));   // 16 bytes on any element

// 8 elements as loaded.
template <typename T>
struct Raw {
    static constexpr int W = (int)sizeof(T) / 2;   // 16-byte vectors
    u32x4_t w[W];
    __device__ __forceinline__ float get(int e) const {
        if constexpr (std::is_same_v<T, float>)
            return __uint_as_float(w[e / 4][e % 4]);
        else if constexpr (std::is_same_v<T, bf16_t>)
            return __uint_as_float(e & 1 ? w[0][e / 2] & 0xFFFF0000u : w[0][e / 2] << 16);
        else
            return (float)__builtin_bit_cast(_Float16, (uint16_t)(e & 1 ? w[0][e / 2] >> 16 : w[0][e / 2]));
    }
    __device__ __forceinline__ void put(int e, T v) {
        if constexpr (std::is_same_v<T, float>) {
            w[e / 4][e % 4] = __float_as_uint(v);
        } else {
            const uint32_t b = __builtin_bit_cast(uint16_t, v);
            w[0][e / 2] = e & 1 ? (w[0][e / 2] & 0xFFFFu) | b << 16 : (w[0][e / 2] & 0xFFFF0000u) | b;
        }
    }
};
// The groups of lane l of a row; 0 past the row's end.  STREAM: the loads leave
// no trace in the caches, as the stores do.  Measured, 262144 x 128 and 16384 x
// 2048: stores so, forward 30.5 -> 26.6 us at 2048; loads so, backward 42 -> 40
// us, but forward 26.6 -> 30.5 us.
template <typename S, bool STREAM, typename T>
__device__ __forceinline__ void load_raw(const T *__restrict__ row, int D, int l, Raw<T> (&v)[S::K]) {
#pragma unroll
    for (int k = 0; k < S::K; ++k) {
        const T *from = row + S::from(l, k, D);
#pragma unroll
        for (int i = 0; i < Raw<T>::W; ++i) v[k].w[i] = u32x4_t{0u, 0u, 0u, 0u};
        if (S::col(l, k) >= D) continue;
        if (S::WHOLE || D >= 8) {
#pragma unroll
            for (int i = 0; i < Raw<T>::W; ++i) {
                const char *p = reinterpret_cast<const char *>(from) + 16 * i;
                if constexpr (!S::WHOLE)
                    v[k].w[i] = *reinterpret_cast<const loose4_t *>(p);
                else if constexpr (STREAM)
                    v[k].w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(p));
                else
                    v[k].w[i] = *reinterpret_cast<const u32x4_t *>(p);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < D) v[k].put(e, from[e]);
        }
    }
}
template <typename S, typename T>
__device__ __forceinline__ void unpack(const Raw<T> (&r)[S::K], float (&v)[S::E]) {
#pragma unroll
    for (int k = 0; k < S::K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * k + e] = r[k].get(e);
}
// fp32 parameters of a lane's groups.
template <typename S>
__device__ __forceinline__ void load_param(const float *__restrict__ p, int D, int l, float (&v)[S::E]) {
    Raw<float> r[S::K];
    load_raw<S, false>(p, D, l, r);
    unpack<S>(r, v);
}
template <typename S, typename T>
__device__ __forceinline__ void store_row(T *__restrict__ row, int D, int l, const float (&v)[S::E]) {
#pragma unroll
    for (int k = 0; k < S::K; ++k) {
        if (S::col(l, k) >= D) continue;
        T *to = row + S::from(l, k, D);
        Raw<T> r;
#pragma unroll
        for (int i = 0; i < Raw<T>::W; ++i) r.w[i] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) r.put(e, round_to<T>(v[8 * k + e]));
        if (S::WHOLE || D >= 8) {
#pragma unroll
            for (int i = 0; i < Raw<T>::W; ++i) {
                char *p = reinterpret_cast<char *>(to) + 16 * i;
                if constexpr (S::WHOLE)
                    __builtin_nontemporal_store(r.w[i], reinterpret_cast<u32x4_t *>(p));
                else
                    *reinterpret_cast<loose4_t *>(p) = r.w[i];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < D) to[e] = round_to<T>(v[8 * k + e]);
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
    if (w) load_param<S>(w, D, l, wv);
    if (b) load_param<S>(b, D, l, bv);
    Raw<x_t> raw[S::K];
    auto load = [&](int64_t r0) { load_raw<S, false>(x + min(r0 + g, rows - 1) * D, D, l, raw); };
    load((int64_t)blockIdx.x * S::ROWS);
    const float n = (float)D;
    for (int64_t r0 = (int64_t)blockIdx.x * S::ROWS; r0 < rows; r0 += (int64_t)gridDim.x * S::ROWS) {
        const int64_t r = r0 + g;
        const bool on = r < rows;
        float v[S::E];
        unpack<S>(raw, v);
        if (r0 + (int64_t)gridDim.x * S::ROWS < rows) load(r0 + (int64_t)gridDim.x * S::ROWS);
        float m = 0.f, q = 0.f, none = 0.f;
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) m += S::WHOLE || S::counts(l, k, e, D) ? v[8 * k + e] : 0.f;
        row_sum2<S>(m, none, s);
        m /= n;
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float &c = v[8 * k + e];
                c -= m;
                q = S::counts(l, k, e, D) ? fmaf(c, c, q) : q;
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

// part: the block's line of partial sums goes to part[block][2][D]; NULL: none
// (the sums are taken all the same: 34 us instead of 38 at 262144 x 128, 41 instead
// of 69 at 2048 x 16384, where the lines are what is saved).
template <typename S, typename x_t, typename y_t>
__global__ __launch_bounds__(S::NT) void layernorm_bwd_kernel(int64_t rows, int D, const y_t *__restrict__ dy,
                                                              const x_t *__restrict__ x,
                                                              const float *__restrict__ mean,
                                                              const float *__restrict__ rstd,
                                                              const float *__restrict__ w, x_t *__restrict__ dx,
                                                              float *__restrict__ part) {
    __shared__ float s[S::NT / 64][2];
    const int l = threadIdx.x % S::L, g = threadIdx.x / S::L;
    // the widest rows' sums leave no registers for a second row
    constexpr bool AHEAD = S::NT < 1024 || S::K == 1;
    float wv[S::E], aw[S::E], ab[S::E];
    if (w) load_param<S>(w, D, l, wv);
    Raw<y_t> ry[S::K];
    Raw<x_t> rx[S::K];
    float rm, rq;
    auto load = [&](int64_t r0) {
        const int64_t r = min(r0 + g, rows - 1);
        load_raw<S, true>(dy + r * D, D, l, ry);
        load_raw<S, true>(x + r * D, D, l, rx);
        rm = mean[r];
        rq = rstd[r];
    };
    load((int64_t)blockIdx.x * S::ROWS);
#pragma unroll
    for (int e = 0; e < S::E; ++e) aw[e] = ab[e] = 0.f;
    const float n = (float)D;
    for (int64_t r0 = (int64_t)blockIdx.x * S::ROWS; r0 < rows; r0 += (int64_t)gridDim.x * S::ROWS) {
        const int64_t r = r0 + g;
        const bool on = r < rows;
        float u[S::E], c[S::E];
        unpack<S>(ry, u);
        unpack<S>(rx, c);
        const float m = rm, q = rq;
        const bool more = r0 + (int64_t)gridDim.x * S::ROWS < rows;
        if (AHEAD && more) load(r0 + (int64_t)gridDim.x * S::ROWS);
        float c1 = 0.f, c2 = 0.f;
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = 8 * k + i;
                c[e] = (c[e] - m) * q;
                if (on && S::counts(l, k, i, D)) {
                    aw[e] = fmaf(u[e], c[e], aw[e]);
                    ab[e] += u[e];
                }
                if (w) u[e] *= wv[e];
                if (S::counts(l, k, i, D)) {
                    c1 += u[e];
                    c2 = fmaf(u[e], c[e], c2);
                }
            }
        row_sum2<S>(c1, c2, s);
        c1 /= n;
        c2 /= n;
#pragma unroll
        for (int e = 0; e < S::E; ++e) u[e] = q * (u[e] - c1 - c[e] * c2);
        if (on) store_row<S>(dx + r * D, D, l, u);
        if (!AHEAD && more) load(r0 + (int64_t)gridDim.x * S::ROWS);
    }
    if (part) {
        // the block's row groups join, a part of the columns at a time
        float *line = part + (int64_t)blockIdx.x * 2 * D;
        if constexpr (S::ROWS == 1) {
#pragma unroll
            for (int k = 0; k < S::K; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int col = S::from(l, k, D) + e;
                    if (S::counts(l, k, e, D)) line[col] = aw[8 * k + e], line[D + col] = ab[8 * k + e];
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
                    const int il = i >> 3, e = i & 7, col = S::from(il, k, D) + e;
                    if (!S::counts(il, k, e, D)) continue;
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

// Adds the lines: COLS columns of the 2 D (weight's, then bias's) by as many
// lanes, 1024 / COLS groups of lines that join in LDS.
template <int COLS>
__global__ __launch_bounds__(1024) void layernorm_sums_kernel(int lines, int D, const float *__restrict__ part,
                                                              float *__restrict__ dw, float *__restrict__ db) {
    constexpr int G = 1024 / COLS;
    __shared__ float s[G][COLS + 1];
    const int c = threadIdx.x % COLS, g = threadIdx.x / COLS, col = blockIdx.x * COLS + c;
    float a = 0.f;
    if (col < 2 * D)
#pragma unroll 8
        for (int i = g; i < lines; i += G) a += part[(int64_t)i * 2 * D + col];
    s[g][c] = a;
    __syncthreads();
    for (int n = G / 2; n >= 1; n >>= 1) {
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

// f(RowShape{}) with the layout for D: 8 elements a lane up to a wave, then two
// or three groups a lane, then more waves; three groups where two would leave
// more than a third of the lanes without any.  The backward pass holds five
// values for each element, so long rows take more lanes instead.
template <bool WHOLE, bool BWD, int NT, typename F>
static hipError_t with_row_shape_of(int D, F f) {
    if (D <= 8) return f(RowShape<1, 1, NT, WHOLE>{});
    if (D <= 16) return f(RowShape<2, 1, NT, WHOLE>{});
    if (D <= 32) return f(RowShape<4, 1, NT, WHOLE>{});
    if (D <= 64) return f(RowShape<8, 1, NT, WHOLE>{});
    if (D <= 128) return f(RowShape<16, 1, NT, WHOLE>{});
    if (D <= 256) return f(RowShape<32, 1, NT, WHOLE>{});
    if (D <= 384) return f(RowShape<16, 3, NT, WHOLE>{});
    if (D <= 512) return f(RowShape<64, 1, NT, WHOLE>{});
    if (D <= 768) return f(RowShape<32, 3, NT, WHOLE>{});
    if (D <= 1024) return f(RowShape<64, 2, NT, WHOLE>{});
    if constexpr (BWD) {
        if (D <= 2048) return f(RowShape<256, 1, NT, WHOLE>{});
        if (D <= 4096) return f(RowShape<512, 1, 512, WHOLE>{});
        if (D <= 8192) return f(RowShape<1024, 1, 1024, WHOLE>{});
    } else {
        if (D <= 1536) return f(RowShape<64, 3, NT, WHOLE>{});
        if (D <= 2048) return f(RowShape<128, 2, NT, WHOLE>{});
        if (D <= 4096) return f(RowShape<256, 2, NT, WHOLE>{});
        if (D <= 6144) return f(RowShape<256, 3, NT, WHOLE>{});
        if (D <= 8192) return f(RowShape<512, 2, 512, WHOLE>{});
        if (D <= 12288) return f(RowShape<512, 3, 512, WHOLE>{});
    }
    return f(RowShape<1024, 2, 1024, WHOLE>{});
}
template <bool BWD, int NT, typename F>
static hipError_t with_row_shape(int D, F f) {
    return D % 8 == 0 ? with_row_shape_of<true, BWD, NT>(D, f) : with_row_shape_of<false, BWD, NT>(D, f);
}

// Threads of a block.  Measured (backward, bf16) with 256, 512 and 1024: 16384 x
// 2048 53, 43 and 45 us, 262144 x 128 40, 39 and 40, 20000 x 264 17.5, 17.3 and
// 54, 4093 x 1001 in fp16 15.5, 15.7 and 27.
constexpr int kFwdThreads = 256, kBwdThreads = 512;
constexpr int64_t kFwdBlocks = 8192;   // more only load the parameters again

// Blocks of the backward kernel, and so lines of partial sums: four turns of a
// block at least, so that the lines stay small beside the rows, unless that
// leaves less than 128 blocks.  Measured in bf16 with 64, 128 and 256 for that
// limit: 255 x 8200 24.6, 21.2 and 25.1 us, 128 x 16384 28.9, 27.0 and 26.9, 511 x
// 4100 18.1, 18.1 and 18.8, 20000 x 264 17.3, 17.3 and 15.6, 4093 x 1001 and 300 x
// 1001 alike.
static int64_t bwd_blocks(int64_t rows, int rows_per_block, int threads) {
    const int64_t most = 256 * (1024 / threads);   // 1024 threads on each of 256 CUs
    const int64_t turns = (rows + rows_per_block - 1) / rows_per_block;
    return std::min({most, turns, std::max<int64_t>((turns + 3) / 4, 128)});
}

size_t layernorm_bwd_workspace(int64_t rows, int32_t dim) {
    int64_t lines = 0;
    with_row_shape<true, kBwdThreads>(dim, [&](auto s) {
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
        return with_row_shape<false, kFwdThreads>(a.dim, [&](auto s) {
            using S = decltype(s);
            const int64_t need = (a.rows + S::ROWS - 1) / S::ROWS;
            const unsigned blocks = (unsigned)(need < kFwdBlocks ? need : kFwdBlocks);
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
            return with_row_shape<true, kBwdThreads>(a.dim, [&](auto s) {
                using S = decltype(s);
                blocks = bwd_blocks(a.rows, S::ROWS, S::NT);
                auto go = [&](auto *kernel) {
                    kernel<<<(unsigned)blocks, S::NT, 0, st>>>(
                        a.rows, a.dim, static_cast<const y_t *>(a.dy), static_cast<const x_t *>(a.x), a.mean, a.rstd,
                        a.weight, static_cast<x_t *>(a.dx), sums ? part : nullptr);
                    return hipGetLastError();
                };
                return go(layernorm_bwd_kernel<S, x_t, y_t>);
            });
        });
    }
    if (e != hipSuccess || !sums) return e;
    ProfScope prof("gdn_layernorm_sums", st);
    auto add = [&](auto cols) {
        constexpr int C = decltype(cols)::value;
        layernorm_sums_kernel<C><<<(unsigned)((2 * a.dim + C - 1) / C), 1024, 0, st>>>((int)blocks, a.dim, part,
                                                                                  a.dweight, a.dbias);
    };
    // whole cache lines where that leaves enough blocks
    if (a.dim >= 4096) add(std::integral_constant<int, 64>{});
    else add(std::integral_constant<int, 16>{});
    return hipGetLastError();
}

}  // namespace gdn
