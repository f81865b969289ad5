// One token of windowed attention for resident sequences: its key and value go into
// the cache, and the query attends to the rows that the cache then holds.  A ring
// holds just the positions that the query sees, and a softmax does not ask for
// their order, so there is no mask but the number of rows.
//
// Bound by reading the cache.  A block takes a part of the rows of one (sequence,
// key head) for all G query heads of the group, its waves tiles of 32 rows in turn:
// S^T = K Q^T in 16 x 16 matrix-core tiles (K's operand straight from memory, the
// heads as columns), running maximum and sum per head, and O^T += V^T P^T with V
// through a private piece of LDS, read transposed.  8-bit rows are widened to the
// query's type exactly; their scales multiply the scores and the probabilities.
// The waves join in LDS; where a sequence's rows are split over blocks, these leave
// (maximum, sum, O) in the workspace, and a second kernel joins them.
//
// Measured (MI355X, a copy 5.35 TB/s), 16 heads on 4 of 128: 256 sequences of 1029 to 2052
// rows in 8 bits 99 to 103 us (515 MB, 5.1 TB/s), in bf16 181 (997 MB, 5.5); of up to 8192
// rows in 8 bits 375 (2.05 GB, 5.5).  In fp32 372 (1.99 GB, 5.35), heads of 64 208 (0.997
// GB, 4.8: some registers spill); 8-bit heads of 256 207 (1.01 GB, 4.9).  Two sequences of
// up to 65536 rows, fp16, 43 us and 5 for the join (268 MB).  What is left are the first
// loads, behind those of slot and length, and the last blocks.  128 registers, so that four
// blocks fit a CU: with 160 the bf16 case takes 205 us.
#include "gdn_cache.h"
#include "gdn_swa.h"

#include <algorithm>

namespace gdn {

constexpr int kTile = 32;             // rows of a wave's tile
constexpr int kStepWaves = 4;
constexpr int kMaxSplits = 1024;      // parts of a sequence's rows: a lane each in the join

struct StepShape {
    int32_t P, KV, H, G, window, sinks, N, splits, per;   // per: rows of a part
    float c;                          // scale log2(e)
};

// Probabilities are taken times 2^kLift: in fp16 the small ones, which many rows may
// share, would be subnormal or 0.  Their sum has the same factor.
template <typename T>
constexpr float kLift = std::is_same_v<T, _Float16> ? 14.f : 0.f;
constexpr float kLiftUnits = 0x1p14f, kLeastUnit = 0x1p-100f;

// Two neighbouring e4m3 values of a word as two 16-bit values, exact.
template <typename T>
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    float x[4];
    from_e4m3(w, x);
    lo = pack2<T>(x[0], x[1]);
    hi = pack2<T>(x[2], x[3]);
}

// acc += A B, 16 x 16, over one 16-byte chunk of both operands' rows.
template <typename T>
__device__ __forceinline__ void mma16(float4_t &acc, u32x4_t a, u32x4_t b) {
    if constexpr (std::is_same_v<T, bf16_t>) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                     __builtin_bit_cast(bf16x8_t, b), acc, 0, 0, 0);
    } else if constexpr (std::is_same_v<T, _Float16>) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b),
                                                    acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), acc, 0, 0, 0);
    }
}

template <typename T, bool Q8, int D>
__global__ __launch_bounds__(64 * kStepWaves, (Rows<T, D>::RB > 256 ? 2 : 4)) void swa_step_kernel(
    StepShape s, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, char *cache, float *scales,
    const int32_t *__restrict__ lengths, const int32_t *__restrict__ slots, T *__restrict__ o,
    float *__restrict__ parts, int32_t *__restrict__ status) {
    constexpr bool F32 = std::is_same_v<T, float>;
    // fp16 on 8 bits holds neither every scale nor every product of one with a
    // probability: V's weights (probability times scale) count in units of the largest
    // so far, a power of two, of which they are less than two, taken times kLiftUnits
    constexpr bool UNITS = Q8 && std::is_same_v<T, _Float16>;
    constexpr float LIFT = UNITS ? 0.f : kLift<T>;
    constexpr int NT = 64 * kStepWaves, RB = D * (int)sizeof(T);
    constexpr int RC = Q8 ? D : RB;               // bytes of a cache row
    constexpr int NS = RB / 64, ND = D / 16;      // steps of the product over D, tiles along D
    using R = Rows<T, D>;
    __shared__ __align__(16) char s_v[kStepWaves][kTile * RB];   // V tiles; then the waves' O
    __shared__ float s_m[kStepWaves][16], s_l[kStepWaves][16], s_ks[Q8 ? kStepWaves : 1][2 * kTile];
    __shared__ __align__(16) char s_new[2][Q8 ? RC : 16];        // the new token's rows as the cache holds them
    __shared__ float s_newscale[2];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, m = l & 15, hq = l >> 4;
    const int n = blockIdx.x / s.KV, hk = blockIdx.x - n * s.KV, split = blockIdx.y;
    const int rows = s.window + s.sinks;

    if (status && blockIdx.x == 0 && split == 0) {   // the whole call's indices, for the caller
        int bad = 0;
        for (int i = tid; i < s.N; i += NT) {
            const int a = slots ? slots[i] : i;
            if (!slot_in_range(a, s.P)) bad |= 1 << 3;
            if (slots && a >= 0)
                for (int j = 0; j < i; ++j) bad |= (slots[j] == a) << 4;
            if (lengths[i] < 0 || lengths[i] >= kCacheMaxLength) bad |= 1 << 5;
        }
        bad = __syncthreads_or(bad & 8) ? 4 : __syncthreads_or(bad & 16) ? 5 : __syncthreads_or(bad & 32) ? 6 : 0;
        if (tid == 0) status[0] = s.N, status[1] = bad;
    }
    if (n >= s.N) return;                         // no sequences: one block, for the status

    constexpr int L = D / 8;
    const bool second = tid >= L;                 // lanes of the new token's rows: k's, then v's
    Raw8<T> fresh;
    const T *from = (second ? v : k) + ((int64_t)n * s.KV + hk) * D + 8 * (tid % L);
    if (Q8 && tid < 2 * L) fresh.load(from);      // does not depend on the slot
    const int slot = slots ? slots[n] : n, pos = lengths[n];
    int bad = slot < 0 || slot >= s.P || pos < 0 || pos >= kCacheMaxLength;
    const int put = bad ? 0 : cache_row(pos, s.window, s.sinks);
    const int r0 = split * s.per;
    uint2 put8{};
    float putscale = 1.f;
    // The block that reads the new token's row writes it.  In 8 bits it takes it from
    // LDS, as memory may still hold the row that it replaces; else it waits for the
    // store (256 sequences, 2052 rows: 8 bits 106 us so, 112 with the wait; bf16 190,
    // for want of registers, and 181).
    if (tid < 2 * L && put >= r0 && put < r0 + s.per) {
        if constexpr (Q8) {
            float x[8];
            fresh.to_f32(x);
            putscale = e4m3_scale(row_amax<L>(x));
            const float inv = e4m3_inverse(putscale);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= inv;
            put8 = to_e4m3(x);
            *reinterpret_cast<uint2 *>(&s_new[second][8 * (tid % L)]) = put8;
            s_newscale[second] = putscale;
        }
    }
    int twice = 0;                                // another sequence of the call on this slot
    if (slots)
        for (int i = tid; i < s.N; i += NT) twice |= i != n && slots[i] == slot;
    bad |= __syncthreads_or(twice);
    const int live = bad ? 0 : min(pos + 1, rows), r1 = min(r0 + s.per, live);
    const int64_t head = ((int64_t)(bad ? 0 : slot) * s.KV + hk) * rows, side = (int64_t)s.P * s.KV * rows;
    const bool mine = put >= r0 && put < r1;
    if (mine && tid < 2 * L) {
        const int64_t row = head + put + (second ? side : 0);
        if constexpr (Q8) {
            *reinterpret_cast<uint2 *>(cache + row * D + 8 * (tid % L)) = put8;
            if (tid % L == 0) scales[row] = putscale;
        } else {
            fresh.load(from);
            fresh.store_lds(reinterpret_cast<T *>(cache) + row * D + 8 * (tid % L));
        }
    }
    if (!Q8 && mine) __syncthreads();

    // the heads' queries, as columns; heads past the group repeat its last
    const int64_t qat = ((int64_t)n * s.H + hk * s.G + min(m, s.G - 1)) * D;
    u32x4_t qf[NS];
#pragma unroll
    for (int x = 0; x < NS; ++x) {
        // 8 bits, D >= 64: a lane's 16 bytes of a row are two steps' chunks
        const int e = Q8 && D >= 64 && !F32 ? 64 * (x >> 1) + 16 * hq + 8 * (x & 1)
                      : Q8 && F32           ? (D >= 64 ? 64 * (x >> 2) + 16 * hq + 4 * (x & 3) : 8 * hq + 4 * x)
                                            : (32 * x + 8 * hq) / (F32 ? 2 : 1);
        qf[x] = *reinterpret_cast<const u32x4_t *>(q + qat + e);
    }

    float4_t acc[ND];
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) acc[dt] = float4_t{0.f, 0.f, 0.f, 0.f};
    float top = -__builtin_inff(), sum = 0.f, unit = kLeastUnit;
    char *vt = s_v[wave];
    // 16 bytes (8) at byte b of row r of k or v, from LDS where it is the new one
    auto renew = [&](auto &x, int r, int which, int b) {
        if (r == put) x = *reinterpret_cast<const std::remove_reference_t<decltype(x)> *>(&s_new[which][b]);
    };
    const char *kbase = cache + head * RC, *vbase = kbase + side * RC;

    for (int t0 = r0 + wave * kTile; t0 < r1; t0 += kStepWaves * kTile) {
        // V: 16 bytes of a row to a lane; rows that are not there are zeros
        constexpr int VL = RC / 16, VR = 64 / VL, VN = kTile / VR;   // lanes a row, rows a load, loads
        u32x4_t vr[VN];
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int r = t0 + i * VR + l / VL;
            vr[i] = *reinterpret_cast<const u32x4_t *>(vbase + (int64_t)min(r, r1 - 1) * RC + 16 * (l % VL));
            if (r >= r1) vr[i] = u32x4_t{0u, 0u, 0u, 0u};
        }
        const bool newest = Q8 && mine && put >= t0 && put < t0 + kTile;
        if (newest)
#pragma unroll
            for (int i = 0; i < VN; ++i) renew(vr[i], t0 + i * VR + l / VL, 1, 16 * (l % VL));
        float sc[2][4], vs = 1.f;
        if constexpr (Q8) {
            // lane x < 32: scale of K's row, x >= 32: of V's
            const int r = min(t0 + (l & 31), r1 - 1);
            vs = scales[head + r + (l >= 32 ? side : 0)];
            if (newest && r == put) vs = s_newscale[l >= 32];
        }
        float4_t S[2] = {float4_t{0.f, 0.f, 0.f, 0.f}, float4_t{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int kr_row = min(t0 + 16 * a + m, r1 - 1);
            const char *kr = kbase + (int64_t)kr_row * RC;
            if constexpr (!Q8) {
                u32x4_t f[NS];
#pragma unroll
                for (int x = 0; x < NS; ++x) f[x] = *reinterpret_cast<const u32x4_t *>(kr + 64 * x + 16 * hq);
#pragma unroll
                for (int x = 0; x < NS; ++x) mma16<T>(S[a], f[x], qf[x]);
            } else if constexpr (D >= 64) {
                u32x4_t f[D / 64];
#pragma unroll
                for (int x = 0; x < D / 64; ++x) f[x] = *reinterpret_cast<const u32x4_t *>(kr + 64 * x + 16 * hq);
                if (newest)
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) renew(f[x], kr_row, 0, 64 * x + 16 * hq);
#pragma unroll
                for (int x = 0; x < D / 64; ++x) {
                    if constexpr (F32) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            float w[4];
                            from_e4m3(f[x][y], w);
                            mma16<T>(S[a], u32x4_t{__float_as_uint(w[0]), __float_as_uint(w[1]), __float_as_uint(w[2]),
                                                   __float_as_uint(w[3])}, qf[4 * x + y]);
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            u32x4_t w;
                            uint32_t lo, hi;
                            widen<T>(f[x][2 * y], lo, hi);
                            w[0] = lo, w[1] = hi;
                            widen<T>(f[x][2 * y + 1], lo, hi);
                            w[2] = lo, w[3] = hi;
                            mma16<T>(S[a], w, qf[2 * x + y]);
                        }
                    }
                }
            } else {
                uint2 f = *reinterpret_cast<const uint2 *>(kr + 8 * hq);
                if (newest) renew(f, kr_row, 0, 8 * hq);
                if constexpr (F32) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float w[4];
                        from_e4m3(y ? f.y : f.x, w);
                        mma16<T>(S[a], u32x4_t{__float_as_uint(w[0]), __float_as_uint(w[1]), __float_as_uint(w[2]),
                                               __float_as_uint(w[3])}, qf[y]);
                    }
                } else {
                    uint32_t w[4];
                    widen<T>(f.x, w[0], w[1]);
                    widen<T>(f.y, w[2], w[3]);
                    mma16<T>(S[a], u32x4_t{w[0], w[1], w[2], w[3]}, qf[0]);
                }
            }
        }
        // V to LDS as rows of T
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int r = i * VR + l / VL, b = 16 * (l % VL);
            if constexpr (!Q8) {
                *reinterpret_cast<u32x4_t *>(vt + R::chunk_off(r, b / 16)) = vr[i];
            } else if constexpr (F32) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float w[4];
                    from_e4m3(vr[i][e], w);
                    *reinterpret_cast<float4_t *>(vt + R::chunk_off(r, b / 4 + e)) = float4_t{w[0], w[1], w[2], w[3]};
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t w[4];
                    widen<T>(vr[i][2 * e], w[0], w[1]);
                    widen<T>(vr[i][2 * e + 1], w[2], w[3]);
                    *reinterpret_cast<u32x4_t *>(vt + R::chunk_off(r, b / 8 + e)) = u32x4_t{w[0], w[1], w[2], w[3]};
                }
            }
        }
        if constexpr (Q8) {
            s_ks[wave][l] = vs;
            asm volatile("" ::: "memory");
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const float4_t x = *reinterpret_cast<const float4_t *>(&s_ks[wave][16 * a + 4 * hq]);
                const float4_t y = *reinterpret_cast<const float4_t *>(&s_ks[wave][kTile + 16 * a + 4 * hq]);
#pragma unroll
                for (int i = 0; i < 4; ++i) S[a][i] *= x[i], sc[a][i] = y[i];
            }
        }
        asm volatile("" ::: "memory");
        // lane (m, hq): head m, rows 16 a + 4 hq + i
        float big = -__builtin_inff();
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (t0 + 16 * a + 4 * hq + i >= r1) S[a][i] = -__builtin_inff();
                big = fmaxf(big, S[a][i]);
            }
        big = fmaxf(big, __shfl_xor(big, 16, 64));
        big = fmaxf(big, __shfl_xor(big, 32, 64));
        if (__any(big > top)) {
            const float up = fmaxf(top, big), f = top == up ? 1.f : __builtin_amdgcn_exp2f((top - up) * s.c);
            top = up;
            sum *= f;
            if constexpr (UNITS) {
                unit *= f;
            } else {
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) acc[dt] *= f;
            }
        }
        // the largest score itself, subtracted before the scale: no rounding of it counts
        const float base = top == -__builtin_inff() ? 0.f : top;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                S[a][i] = __builtin_amdgcn_exp2f(fmaf(S[a][i] - base, s.c, LIFT));
                sum += S[a][i];
                // the scale joins before the rounding; a row that is not there has none
                if constexpr (Q8)
                    S[a][i] = t0 + 16 * a + 4 * hq + i < r1 ? S[a][i] * sc[a][i] : 0.f;
            }
        if constexpr (UNITS) {
            float most = fmaxf(unit, kLeastUnit);
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) most = fmaxf(most, S[a][i]);
            most = fmaxf(most, __shfl_xor(most, 16, 64));
            most = fmaxf(most, __shfl_xor(most, 32, 64));
            most = __uint_as_float(__float_as_uint(most) & 0x7F800000u);
            const float inv = e4m3_inverse(most);
            if (__any(most != unit)) {
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) acc[dt] *= unit * inv;
            }
            unit = most;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[a][i] *= inv * kLiftUnits;
        }
        if constexpr (F32) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 16 * a + 4 * hq + i;
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) {
                        const float w =
                            *reinterpret_cast<const float *>(vt + R::chunk_off(r, 4 * dt + (m >> 2)) + 4 * (m & 3));
                        acc[dt] = __builtin_amdgcn_mfma_f32_16x16x4f32(w, S[a][i], acc[dt], 0, 0, 0);
                    }
                }
        } else {
            u32x4_t p;
#pragma unroll
            for (int a = 0; a < 2; ++a) p[2 * a] = pack2<T>(S[a][0], S[a][1]), p[2 * a + 1] = pack2<T>(S[a][2], S[a][3]);
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) {
                const int r = 4 * hq + (m >> 2);
                const char *f = vt + R::chunk_off(r, 2 * dt + ((m & 3) >> 1)) + 8 * (m & 1);
                const uint2 lo = lds_read_tr16(f), hi = lds_read_tr16(f + 16 * RB);
                mma16<T>(acc[dt], u32x4_t{lo.x, lo.y, hi.x, hi.y}, p);
            }
        }
        asm volatile("" ::: "memory");            // the next tile's V is written behind these reads
    }

    if constexpr (UNITS)
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) acc[dt] *= unit / kLiftUnits;

    // the waves join
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    __syncthreads();
    if (hq == 0) s_m[wave][m] = top, s_l[wave][m] = sum;
    float *own_o = reinterpret_cast<float *>(vt);   // [16 heads][D], half of a 16-bit V tile's rows
#pragma unroll
    for (int dt = 0; dt < ND; ++dt)
        *reinterpret_cast<float4_t *>(own_o + m * D + 16 * dt + 4 * hq) = acc[dt];
    __syncthreads();
    const int64_t out = ((int64_t)n * s.H + hk * s.G) * D;
    const bool whole = s.splits == 1;
    float *to = parts + (((int64_t)n * s.KV + hk) * s.splits + split) * (int64_t)s.G * (D + 2);
    for (int i = tid; i < s.G * D; i += NT) {
        const int g = i / D;
        float up = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < kStepWaves; ++w) up = fmaxf(up, s_m[w][g]);
        const float base = up == -__builtin_inff() ? 0.f : up;
        float x = 0.f, z = 0.f;
#pragma unroll
        for (int w = 0; w < kStepWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f((s_m[w][g] - base) * s.c);
            z += f * s_l[w][g];
            x += f * reinterpret_cast<const float *>(s_v[w])[i];
        }
        if (whole) {
            o[out + i] = round_to<T>(z == 0.f ? 0.f : x / z);
        } else {
            to[2 * s.G + i] = x;
            if (i % D == 0) to[2 * g] = up, to[2 * g + 1] = z;
        }
    }
}

// Joins the parts of one (sequence, query head): groups of D lanes take the parts in
// turn and join in LDS, in a fixed order.
template <typename T, int D>
__global__ __launch_bounds__(1024) void swa_step_join_kernel(StepShape s, const float *__restrict__ parts,
                                                             T *__restrict__ o) {
    __shared__ float s_w[kMaxSplits], s_x[1024], s_m[16], s_z[16];
    const int tid = threadIdx.x, g = blockIdx.x % s.G, unit = blockIdx.x / s.G, n = unit / s.KV, hk = unit - n * s.KV;
    const int nt = blockDim.x, waves = (nt + 63) / 64, groups = nt / D;
    const int64_t step = (int64_t)s.G * (D + 2);
    const float *from = parts + (int64_t)unit * s.splits * step + 2 * g;
    float up = -__builtin_inff(), z = 0.f, x = 0.f;
    for (int p = tid; p < s.splits; p += nt) up = fmaxf(up, from[p * step]);
    for (int d = 32; d >= 1; d >>= 1) up = fmaxf(up, __shfl_xor(up, d, 64));
    if ((tid & 63) == 0) s_m[tid >> 6] = up;
    __syncthreads();
    for (int w = 0; w < waves; ++w) up = fmaxf(up, s_m[w]);
    const float base = up == -__builtin_inff() ? 0.f : up;
    for (int p = tid; p < s.splits; p += nt) {
        const float f = __builtin_amdgcn_exp2f((from[p * step] - base) * s.c);
        s_w[p] = f;
        z = fmaf(f, from[p * step + 1], z);
    }
    for (int d = 32; d >= 1; d >>= 1) z += __shfl_xor(z, d, 64);
    if ((tid & 63) == 0) s_z[tid >> 6] = z;
    __syncthreads();
    z = 0.f;
    for (int w = 0; w < waves; ++w) z += s_z[w];
    const int d = tid % D, q = tid / D;
    from += 2 * (s.G - g) + g * D + d;
#pragma unroll 8
    for (int p = q; p < s.splits; p += groups) x = fmaf(s_w[p], from[p * step], x);
    s_x[tid] = x;
    __syncthreads();
    if (q) return;
    x = 0.f;
    for (int i = 0; i < groups; ++i) x += s_x[i * D + d];
    o[((int64_t)n * s.H + hk * s.G + g) * D + d] = round_to<T>(z == 0.f ? 0.f : x / z);
}

// Enough blocks for the GPU, each with a tile for every wave at least.  Measured for
// 1024, 2048 and 4096 blocks, kernel and join: 256 sequences above 113, 142 and 157 us
// (no join with 1024), 64 sequences 42, 51 and 61, 16 sequences 24 each, two of 65536 rows
// 64, 68 and 73.
int swa_step_splits(const SwaStepArgs &a) {
    const int64_t rows = (int64_t)a.c.window + a.c.sinks, units = std::max<int64_t>((int64_t)a.c.N * a.c.KV, 1);
    const int64_t most = std::max<int64_t>(rows / (kStepWaves * kTile), 1);
    return (int)std::max<int64_t>(std::min<int64_t>(1024 / units, std::min<int64_t>(most, kMaxSplits)), 1);
}

size_t swa_step_workspace(const SwaStepArgs &a) {
    const int splits = swa_step_splits(a);
    return splits == 1 ? 0 : (size_t)a.c.N * splits * a.H * (a.c.D + 2) * 4;
}

hipError_t launch_swa_step(const SwaStepArgs &a, hipStream_t st) {
    const CacheArgs &c = a.c;
    StepShape s{};
    s.P = c.P, s.KV = c.KV, s.H = a.H, s.G = a.H / c.KV, s.window = c.window, s.sinks = c.sinks, s.N = c.N;
    s.splits = swa_step_splits(a);
    const int64_t rows = (int64_t)c.window + c.sinks;
    s.per = (int)(((rows + s.splits - 1) / s.splits + kTile - 1) / kTile * kTile);
    s.c = a.scale * 1.4426950408889634f;
    float *parts = static_cast<float *>(a.workspace);
    auto go = [&](auto t, auto q8, auto dim) {
        using T = decltype(t);
        constexpr int D = decltype(dim)::value;
        {
            ProfScope prof("gdn_swa_step", st);
            swa_step_kernel<T, decltype(q8)::value, D><<<dim3(std::max(c.N * c.KV, 1), s.splits), 64 * kStepWaves,
                                                              0, st>>>(
                s, static_cast<const T *>(a.q), static_cast<const T *>(c.k), static_cast<const T *>(c.v),
                static_cast<char *>(c.cache), c.scales, c.lengths, c.slots, static_cast<T *>(a.o), parts, c.status);
        }
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || s.splits == 1 || c.N == 0) return e;
        ProfScope prof("gdn_swa_step_join", st);
        // eight parts to a group of lanes
        const int nt = std::max(D * std::max(std::min((s.splits + 7) / 8, 1024 / D), 1), 64);
        swa_step_join_kernel<T, D><<<c.N * a.H, nt, 0, st>>>(s, parts, static_cast<T *>(a.o));
        return hipGetLastError();
    };
    return swa_with<true>(c.dtype, c.D, [&](auto t, auto dim) {
        return c.cache_dtype == DT_E4M3 ? go(t, std::true_type{}, dim) : go(t, std::false_type{}, dim);
    });
}

}  // namespace gdn
