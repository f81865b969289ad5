// The resident cache of windowed attention, written and read back:
//   position p of a sequence sits in row p (p < sinks), else sinks + (p - sinks) mod window
// Rows are moved whole, in the cache's own type or as e4m3 with a power of two
// per row (gdn_cache.h).  Both directions are bound by HBM.
//
// Every block checks lengths, slots and offsets itself (a few KiB, in L2), so a bad
// one makes all of them write nothing without a second launch; the same pass sums
// up how many rows each sequence moves.  The rows of all sequences, each with its
// heads, are one list, of which a block takes a contiguous piece: a group of
// D / 8 lanes takes a row at a time, and follows the sequences as it goes.
// Writing, only what stays is touched: of the tokens of one call the last `window`
// and those that are sinks, so no two tokens write one row.
#include "gdn_cache.h"

#include <algorithm>

namespace gdn {

constexpr int kThreads = 256;

struct CacheShape {
    int32_t P, KV, window, sinks, N, tokens, per_seq;   // per_seq: tokens of a row, not packed
};

template <typename T, bool Q8, bool READ, int L>
__global__ __launch_bounds__(kThreads) void cache_rows_kernel(CacheShape s, const int32_t *__restrict__ lengths,
                                                             const int32_t *__restrict__ slots,
                                                             const int32_t *__restrict__ cu, T *__restrict__ k,
                                                             T *__restrict__ v, void *__restrict__ cache,
                                                             float *__restrict__ scales,
                                                             int32_t *__restrict__ status) {
    constexpr int D = 8 * L, GROUPS = kThreads / L, U = 4;
    extern __shared__ int first[];               // rows moved by the sequences before: N + 1
    __shared__ int part[kThreads / 64], s_code;
    __shared__ uint32_t seen[kCacheMaxSlots / 32];
    const int tid = threadIdx.x, rows = s.window + s.sinks;
    if (slots)
        for (int i = tid; i < (s.P + 31) / 32; i += kThreads) seen[i] = 0u;
    if (tid == 0) s_code = 0, first[0] = 0;
    __syncthreads();
    int bad = 0, total = 0;
    if (cu && tid == 0) bad |= (cu[0] != 0) << 0 | (cu[s.N] != s.tokens) << 2;
    for (int n0 = 0; n0 < s.N; n0 += kThreads) {
        const int n = n0 + tid;
        int x = 0;
        if (n < s.N) {
            const int c0 = cu ? cu[n] : 0, len = cu ? cu[n + 1] - c0 : s.per_seq, have = lengths ? lengths[n] : 0;
            const int slot = slots ? slots[n] : n;
            if (cu && cu[n + 1] < c0) bad |= 1 << 1;
            if (!slot_in_range(slot, s.P))
                bad |= 1 << 3;
            else if (slots && slot >= 0 && (atomicOr(&seen[slot >> 5], 1u << (slot & 31)) >> (slot & 31) & 1u))
                bad |= 1 << 4;
            if (have < 0 || have >= kCacheMaxLength || (!READ && (int64_t)have + len >= kCacheMaxLength)) bad |= 1 << 5;
            if (READ) {
                x = min(have, rows);
                if (slot >= 0 && x > len) bad |= 1 << 6;
            } else {
                x = min(len, s.window) + max(min(s.sinks, have + len - s.window) - have, 0);
            }
            if (slot < 0 || bad) x = 0;
        }
        int sum = x;
        for (int d = 1; d < 64; d <<= 1) {
            const int y = __shfl_up(sum, d, 64);
            if ((tid & 63) >= d) sum += y;
        }
        if ((tid & 63) == 63) part[tid >> 6] = sum;
        __syncthreads();
        sum += total;
        for (int w = 0; w < kThreads / 64; ++w) {
            if (w < (tid >> 6)) sum += part[w];
            total += part[w];
        }
        if (n < s.N) first[n + 1] = sum;
        __syncthreads();
    }
    if (bad) atomicOr(&s_code, bad);
    __syncthreads();
    bad = s_code;
    if (status && blockIdx.x == 0 && tid == 0) {
        status[0] = s.N;
        status[1] = bad ? __builtin_ctz(bad) + 1 : 0;
    }
    if (bad) return;

    // rows of k, then the same of v
    const int64_t half = (int64_t)total * s.KV, all = 2 * half;
    const int64_t turn = (int64_t)GROUPS * U, per = ((all + gridDim.x - 1) / gridDim.x + turn - 1) / turn * turn;
    const int64_t begin = blockIdx.x * per, end = min(begin + per, all);
    const int g = tid / L, l = tid % L;
    int n = -1, side = 0;
    for (int64_t i0 = begin; i0 < end; i0 += turn) {
        float x[U][8];
        int64_t to[U], row_at[U];                // elements of k or v, rows of the cache
        int sides[U];
        float scale[U];
        u32x4_t raw[U][sizeof(T) / 2];
        uint2 raw8[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + (int64_t)u * GROUPS + g;
            to[u] = -1;
            scale[u] = 0.f;
            if (i >= end) continue;
            const int sd = i >= half;
            const int64_t item = i - (sd ? half : 0);
            const int r = (int)(item / s.KV), h = (int)(item - (int64_t)r * s.KV);
            if (n < 0 || sd != side || r < first[n]) {
                int a = 0, b = s.N;              // the last sequence whose first row is at most r
                while (b - a > 1) {
                    const int c = (a + b) / 2;
                    if (first[c] <= r) a = c;
                    else b = c;
                }
                n = a, side = sd;
            }
            while (first[n + 1] <= r) ++n;
            const int o = r - first[n], have = lengths ? lengths[n] : 0, slot = slots ? slots[n] : n;
            const int64_t t0 = cu ? cu[n] : (int64_t)n * s.per_seq;
            int t, row;
            if (READ) {
                t = o;
                row = have <= rows || o < s.sinks
                          ? o
                          : cache_row(have - s.window + (o - s.sinks), s.window, s.sinks);
            } else {
                const int len = (cu ? cu[n + 1] : (int)(t0 + s.per_seq)) - (int)t0, tail = min(len, s.window);
                const int head = first[n + 1] - first[n] - tail;
                t = o < head ? o : len - tail + (o - head);
                row = cache_row(have + t, s.window, s.sinks);
            }
            to[u] = ((t0 + t) * s.KV + h) * D;
            row_at[u] = (((int64_t)sd * s.P + slot) * s.KV + h) * rows + row;
            sides[u] = sd;
            if (READ) {
                if constexpr (Q8) {
                    raw8[u] = *reinterpret_cast<const uint2 *>(static_cast<const char *>(cache) + row_at[u] * D + 8 * l);
                    scale[u] = scales[row_at[u]];
                } else {
#pragma unroll
                    for (int e = 0; e < (int)sizeof(T) / 2; ++e)
                        raw[u][e] = *reinterpret_cast<const u32x4_t *>(
                            static_cast<const char *>(cache) + (row_at[u] * D + 8 * l) * (int64_t)sizeof(T) + 16 * e);
                }
            } else {
                const T *from = (sd ? v : k) + to[u] + 8 * l;
#pragma unroll
                for (int e = 0; e < (int)sizeof(T) / 2; ++e)
                    raw[u][e] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(from) + e);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (READ) {
                T *out = (sides[u] ? v : k) + to[u] + 8 * l;
                if constexpr (Q8) {
                    if (to[u] < 0) continue;
                    float a[4], b[4];
                    from_e4m3(raw8[u].x, a);
                    from_e4m3(raw8[u].y, b);
                    T y[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = round_to<T>(a[e] * scale[u]), y[4 + e] = round_to<T>(b[e] * scale[u]);
                    u32x4_t w[sizeof(T) / 2];
                    __builtin_memcpy(w, y, sizeof(w));
#pragma unroll
                    for (int e = 0; e < (int)sizeof(T) / 2; ++e)
                        __builtin_nontemporal_store(w[e], reinterpret_cast<u32x4_t *>(out) + e);
                } else {
                    if (to[u] < 0) continue;
#pragma unroll
                    for (int e = 0; e < (int)sizeof(T) / 2; ++e)
                        __builtin_nontemporal_store(raw[u][e], reinterpret_cast<u32x4_t *>(out) + e);
                }
            } else if constexpr (Q8) {
                T y[8];
                __builtin_memcpy(y, raw[u], sizeof(y));
#pragma unroll
                for (int e = 0; e < 8; ++e) x[u][e] = to[u] < 0 ? 0.f : to_f32(y[e]);
                const float sc = e4m3_scale(row_amax<L>(x[u])), inv = e4m3_inverse(sc);
                if (to[u] < 0) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[u][e] *= inv;
                *reinterpret_cast<uint2 *>(static_cast<char *>(cache) + row_at[u] * D + 8 * l) = to_e4m3(x[u]);
                if (l == 0) scales[row_at[u]] = sc;
            } else {
                if (to[u] < 0) continue;
#pragma unroll
                for (int e = 0; e < (int)sizeof(T) / 2; ++e)
                    *reinterpret_cast<u32x4_t *>(static_cast<char *>(cache) +
                                                 (row_at[u] * D + 8 * l) * (int64_t)sizeof(T) + 16 * e) = raw[u][e];
            }
        }
    }
}

template <bool READ>
static hipError_t launch_cache(const CacheArgs &a, hipStream_t st) {
    ProfScope prof(READ ? "gdn_cache_read" : "gdn_cache_write", st);
    CacheShape s{a.P, a.KV, a.window, a.sinks, a.N, a.tokens, a.cu ? 0 : a.tokens / std::max(a.N, 1)};
    const int64_t rows = (int64_t)a.window + a.sinks;
    const int64_t most = 2 * a.KV * (READ ? std::min<int64_t>(a.N * rows, a.tokens)
                                          : std::min<int64_t>(a.N * rows, a.tokens));
    const size_t lds = 4 * ((size_t)a.N + 1);
    auto with_lanes = [&](auto t, auto q8, auto lanes) {
        using T = decltype(t);
        constexpr int L = decltype(lanes)::value;
        const int64_t turns = (most + kThreads / L * 4 - 1) / (kThreads / L * 4);
        const unsigned blocks = (unsigned)std::max<int64_t>(std::min<int64_t>(turns, 2048), 1);
        cache_rows_kernel<T, decltype(q8)::value, READ, L><<<blocks, kThreads, lds, st>>>(
            s, a.lengths, a.slots, a.cu, static_cast<T *>(const_cast<void *>(a.k)),
            static_cast<T *>(const_cast<void *>(a.v)), a.cache, a.scales, a.status);
        return hipGetLastError();
    };
    auto with_type = [&](auto t, auto q8) {
        switch (a.D) {
            case 32: return with_lanes(t, q8, std::integral_constant<int, 4>{});
            case 64: return with_lanes(t, q8, std::integral_constant<int, 8>{});
            case 128: return with_lanes(t, q8, std::integral_constant<int, 16>{});
        }
        return with_lanes(t, q8, std::integral_constant<int, 32>{});
    };
    if (a.cache_dtype == DT_E4M3) {
        if (a.dtype == DT_BF16) return with_type(bf16_t{}, std::true_type{});
        if (a.dtype == DT_FP16) return with_type(_Float16{}, std::true_type{});
        return with_type(float{}, std::true_type{});
    }
    // moved as they are: by size alone
    if (a.dtype == DT_FP32) return with_type(float{}, std::false_type{});
    return with_type(bf16_t{}, std::false_type{});
}

hipError_t launch_cache_write(const CacheArgs &a, hipStream_t st) { return launch_cache<false>(a, st); }
hipError_t launch_cache_read(const CacheArgs &a, hipStream_t st) { return launch_cache<true>(a, st); }

}  // namespace gdn
