// The resident cache of windowed attention, written and read back:
//   position p of a sequence sits in row p (p < sinks), else sinks + (p - sinks) mod window
// Rows are moved whole, in the cache's own type or as e4m3 with a power of two
// per row (gdn_cache.h).  Both directions are bound by HBM.  Measured (MI355X, a copy of
// 2 GiB 4.84 TB/s): 256 sequences' 8-bit rows read back to bf16, 4 heads of 128, 317 us
// (1.5 GB, 4.7 TB/s); 64 prompts' last rows written in 8 bits 54 us (246 MB, 4.6), 2386
// tokens of 256 sequences in bf16 8 to 9 us, most of it the look at the indices.  In
// the inputs' own type: the 256 sequences' rows read back in bf16 399 us (1.98 GB, 5.0
// TB/s), in fp32 890 (3.96 GB, 4.4); the prompts' rows written in bf16 67 (325 MB, 4.8),
// in fp32 150 (650 MB, 4.3).
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

    // Rows of k with their heads, then the same of v; the rows of a block's piece go by
    // its groups in turn.  A group keeps where it is, so that a step is some additions.
    const int64_t all = 2 * (int64_t)total * s.KV;
    const int64_t turn = (int64_t)GROUPS * U, per = ((all + gridDim.x - 1) / gridDim.x + turn - 1) / turn * turn;
    const int64_t begin = blockIdx.x * per, end = min(begin + per, all);
    if (begin >= end) return;
    const int g = tid / L, l = tid % L;
    const int step_r = GROUPS / s.KV, step_h = GROUPS - step_r * s.KV;
    int64_t left = end - begin - g;                // items from this one on
    int64_t at = (begin + g) / s.KV;               // row of both sides
    int h = (int)(begin + g - at * s.KV), side = at >= total, r = (int)(at - (side ? total : 0));
    int n = s.N, next = 0;                         // the sequence of row r, and the first row of the next
    int tokens0 = 0, head = 0, jump = 0, ring = 0; // its first token; rows that are not of the ring's run
    int64_t page = 0;                              // its first row in the cache
    auto enter = [&]() {
        int a = 0, b = s.N;                        // the last sequence whose first row is at most r
        while (b - a > 1) {
            const int c = (a + b) / 2;
            if (first[c] <= r) a = c;
            else b = c;
        }
        n = a;
        while (first[n + 1] <= r) ++n;
        next = first[n + 1];
        const int have = lengths ? lengths[n] : 0, slot = slots ? slots[n] : n;
        tokens0 = cu ? cu[n] : n * s.per_seq;
        page = ((int64_t)side * s.P + slot) * s.KV * rows;
        if (READ) {
            // rows o < head stand as they are, row o >= head at ring place (ring + o) mod window
            head = have <= rows ? rows : s.sinks;
            ring = have <= rows ? 0 : (have - s.window - s.sinks) % s.window - s.sinks;
            jump = 0;
        } else {
            // the first `head` tokens are sinks, then `jump` tokens are passed over
            const int len = (cu ? cu[n + 1] : tokens0 + s.per_seq) - tokens0, tail = min(len, s.window);
            head = next - first[n] - tail;
            jump = len - tail - head;
            const int start = have + len - tail - s.sinks;
            ring = (start > 0 ? start % s.window : start) - head;
        }
    };
    for (; __any(left > 0); left -= turn) {
        float x[U][8];
        int64_t to[U], row_at[U];                  // elements of k or v, rows of the cache
        int sides[U];
        float scale[U];
        u32x4_t raw[U][sizeof(T) / 2];
        uint2 raw8[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            to[u] = -1;
            scale[u] = 0.f;
            if (left - (int64_t)u * GROUPS <= 0) continue;
            if (n == s.N || r >= next) enter();
            const int o = r - first[n], t = READ ? o : o < head ? o : o + jump;
            int row;
            if (READ) {
                int x0 = ring + o;
                if (x0 >= s.window) x0 -= s.window;
                row = o < head ? o : s.sinks + x0;
            } else {
                // tokens before the ring's rows are sinks, in their own rows; ring + o < 0 too
                int x0 = ring + o;
                if (x0 >= s.window) x0 -= s.window;
                row = o < head ? (lengths ? lengths[n] : 0) + o : s.sinks + x0;
            }
            to[u] = (((int64_t)tokens0 + t) * s.KV + h) * D;
            row_at[u] = page + (int64_t)h * rows + row;
            sides[u] = side;
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
                const T *from = (side ? v : k) + to[u] + 8 * l;
#pragma unroll
                for (int e = 0; e < (int)sizeof(T) / 2; ++e)
                    raw[u][e] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(from) + e);
            }
            h += step_h;
            r += step_r;
            if (h >= s.KV) h -= s.KV, ++r;
            if (r >= total) r -= total, ++side, n = s.N;
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
    const int64_t most = 2 * a.KV * std::min<int64_t>(a.N * rows, a.tokens);
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
