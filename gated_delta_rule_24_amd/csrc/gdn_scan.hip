// Gated linear recurrence h_t = alpha_t h_{t-1} + x_t per channel, its
// gradient and its single step.  All three are bound by HBM: no value is used
// twice, and a token costs one exp and two or three multiply-adds a channel.
//
// Sequences in one pass.  Tokens compose as affine maps h -> A h + H:
//   (A1, H1) then (A2, H2)  =  (A1 A2, A2 H1 + H2).
// A block takes a tile of kTc tokens x 64 channels, reads it once into
// registers, forms its threads' maps, joins them in LDS, gets the state that
// enters the tile, runs the recurrence from the registers and writes the
// result: every tensor crosses HBM once, whatever the length.  The state that
// enters a tile comes from the tiles before it in the same chain (batch row
// and channel tile):
//   - each tile publishes its own map (agg) as soon as it has it;
//   - a chain's tiles form groups of kGroup; the last tile of a group
//     publishes the state that leaves the group (pre);
//   - a tile takes the state that enters its group and applies the maps of
//     the tiles before it in the group, in order.  The order of every sum is
//     fixed, so equal calls give equal bits, and only one hand-over per
//     kGroup tiles is serial.
// Every published value is one 8-byte word, written and read by relaxed
// device-scope atomics, so a word is whole or not there: scan_setup_kernel
// fills the words with kEmpty, which no published word equals (not-a-number
// is published in one form).  No fence is needed, as nothing but the word
// itself is handed over.
// Every wait ends: a block draws its place in its chain from the chain's
// counter when it turns to a tile, so it waits only for tiles that were begun
// before its own, and the first of a chain waits for none.  Should two calls
// run on one workspace at once, against the contract, a wait gives up after
// kPatience looks (about a second; a wait in earnest takes microseconds): the
// state is then not-a-number and the workspace's code 4.
//
// The gradient is the same recurrence backwards in e_t = alpha_t g_t,
//   g_t = dh_t + e_{t+1},  e_t = alpha_t g_t,
// with dx_t = g_t, dlog_alpha_t = e_t h_{t-1}.
//
// Packed batches are one chain over all tokens, cut at sequence starts: a map
// that crosses a start forgets what enters it.  Such a map has A = -0 (no
// product of exponentials is negative), and forgetting is a selection, not a
// product with zero, so not-a-number and infinite states stay in their own
// sequence.
#include "gdn_device.h"
#include "gdn_ops.h"
#include "gdn_types.h"

namespace gdn {

constexpr int kTc = 128;        // tokens of a tile
constexpr int kCw = 64;         // channels of a tile
constexpr int kElems = kTc * kCw / 256;   // elements per thread
constexpr int kGroup = 8;       // tiles per group of a chain
constexpr uint64_t kEmpty = ~0ull;
constexpr int64_t kMaxBlocks = 1 << 22;
constexpr int kPatience = 1 << 20;

static int64_t scan_tiles(int64_t n, int w) { return (n + w - 1) / w; }

ScanWorkspace scan_workspace_layout(int32_t B, int32_t T, int32_t D, int32_t N, bool packed) {
    ScanWorkspace w;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    w.rows = packed ? 1 : B;
    w.chunks = scan_tiles(T, kTc);
    w.tiles = scan_tiles(D, kCw);
    const bool chained = w.chunks > 1;
    const int64_t words = chained ? w.rows * w.tiles * kCw : 0;
    size_t at = 256;                                   // meta
    w.off_tab = at;
    at += packed ? up((size_t)(w.chunks + 1) * 4) : 0;
    w.off_ctr = at;
    at += chained ? up((size_t)w.rows * w.tiles * 4) : 0;
    w.off_agg = at;
    at += up((size_t)words * w.chunks * 8);
    w.off_pre = at;
    at += up((size_t)words * scan_tiles(w.chunks, kGroup) * 8);
    w.total = at;
    return w;
}

// Empties the words, zeroes the counters; packed: checks cu_seqlens (codes as
// in chunk_table_kernel) and finds, for each tile of tokens, the first offset
// that is not before it.
__global__ __launch_bounds__(256) void scan_setup_kernel(int N, int T, int nchunk, const int32_t *__restrict__ cu,
                                                         int32_t *__restrict__ meta, int32_t *__restrict__ tab,
                                                         int32_t *__restrict__ ctr, int64_t nctr,
                                                         u32x4_t *__restrict__ words, int64_t nwords16) {
    const int64_t tid = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)gridDim.x * 256;
    for (int64_t i = tid; i < nwords16; i += all) words[i] = u32x4_t{~0u, ~0u, ~0u, ~0u};
    for (int64_t i = tid; i < nctr; i += all) ctr[i] = 0;
    if (cu) {
        for (int64_t c = tid; c < nchunk; c += all) {
            const int64_t t0 = c * kTc;
            int lo = 0, hi = N;            // the first n with cu[n] >= t0 (N if there is none)
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] < t0) lo = mid + 1;
                else hi = mid;
            }
            tab[c] = lo;
        }
        if (blockIdx.x == 0) {
            __shared__ int s_code;
            if (threadIdx.x == 0) s_code = 0;
            __syncthreads();
            int code = 0;
            for (int n = threadIdx.x; n <= N; n += 256) {
                const int v = cu[n];
                if (n == 0 && v != 0) code |= 1;
                if (n > 0 && cu[n - 1] > v) code |= 2;
                if (n == N && v != T) code |= 4;
            }
            if (code) atomicOr(&s_code, code);
            __syncthreads();
            if (threadIdx.x == 0) {
                meta[0] = nchunk;
                meta[1] = (s_code & 1) ? 1 : ((s_code & 2) ? 2 : (s_code ? 3 : 0));
            }
        }
    }
}

// ---- maps ---------------------------------------------------------------------

__device__ __forceinline__ bool forgets(float A) { return __float_as_uint(A) == 0x80000000u; }
// What map (A, H) makes of state s.
template <bool PACKED>
__device__ __forceinline__ float apply(float A, float H, float s) {
    const float v = fmaf(A, s, H);
    return PACKED && forgets(A) ? H : v;
}
// The word of a published pair.  H is not-a-number in one form only, so no
// word equals kEmpty.
__device__ __forceinline__ uint64_t word(float A, float H) {
    const uint32_t h = H != H ? 0x7FC00000u : __float_as_uint(H);
    return ((uint64_t)__float_as_uint(A) << 32) | h;
}
__device__ __forceinline__ void put(uint64_t *p, uint64_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get(const uint64_t *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// exp(x): exp2's instruction on x log2(e).
__device__ __forceinline__ float exp_gate(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// V consecutive elements as loaded.
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, T (&o)[V]) {
    struct alignas(sizeof(T) * V) A {
        T e[V];
    };
    const A a = *reinterpret_cast<const A *>(p);
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = a.e[j];
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const T (&v)[V]) {
    struct alignas(sizeof(T) * V) A {
        T e[V];
    };
    A a;
#pragma unroll
    for (int j = 0; j < V; ++j) a.e[j] = v[j];
    *reinterpret_cast<A *>(p) = a;
}

// ---- the chain --------------------------------------------------------------------

struct Chain {
    int T, D, N, nchunk, ntile;
    int64_t nchain, blocks;        // chains, tiles of all chains
    const int32_t *cu;
    int32_t *meta;
    const int32_t *tab;
    int32_t *ctr;
    uint64_t *agg, *pre;
};

// The state entering tile `k` (its place in the chain) for column `c`, from
// the tile's own map: waits for the tiles before it and publishes what the
// tiles after it need.  Returns the state that enters; `first` is the state
// that enters the chain.
template <bool PACKED>
__device__ __forceinline__ float chain_state(const Chain &p, int64_t chain, int k, int c, float A, float H,
                                             float first) {
    if (p.nchunk == 1) return first;
    const int64_t pitch = (int64_t)kCw;
    const int r = k / kGroup, s = k % kGroup;
    uint64_t *agg = p.agg + (chain * p.nchunk + r * kGroup) * pitch + c;
    uint64_t *pre = p.pre + (chain * ((p.nchunk + kGroup - 1) / kGroup) + r) * pitch + c;
    const bool more = k + 1 < p.nchunk;
    if (more && s < kGroup - 1) put(agg + s * pitch, word(A, H));
    float in = first;
    if (k > 0) {
        uint64_t w[kGroup];
        for (int looks = 0;; ++looks) {
            bool all = true;
#pragma unroll
            for (int j = 0; j < kGroup - 1; ++j) w[j] = j < s ? get(agg + j * pitch) : 0;
            w[kGroup - 1] = r > 0 ? get(pre) : 0;
#pragma unroll
            for (int j = 0; j < kGroup; ++j) all = all && w[j] != kEmpty;
            if (__all(all)) break;
            if (looks >= kPatience) {      // kEmpty's halves are not-a-number
                p.meta[1] = 4;
                break;
            }
            __builtin_amdgcn_s_sleep(1);
        }
        if (r > 0) in = __uint_as_float((uint32_t)w[kGroup - 1]);
#pragma unroll
        for (int j = 0; j < kGroup - 1; ++j)
            if (j < s) in = apply<PACKED>(__uint_as_float((uint32_t)(w[j] >> 32)), __uint_as_float((uint32_t)w[j]), in);
    }
    if (more && s == kGroup - 1) put(pre + pitch, word(0.f, apply<PACKED>(A, H, in)));
    return in;
}

// Whole-number division, in 32 bits where that is enough.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t modulo(int64_t a, int64_t b) { return a - quotient(a, b) * b; }

// The place of the block's next tile in its chain.
__device__ __forceinline__ int draw_place(const Chain &p, int64_t chain, int *s_k) {
    if (p.nchunk <= 1) return 0;
    if (threadIdx.x == 0) *s_k = atomicAdd(&p.ctr[chain], 1);
    __syncthreads();
    return *s_k;
}

// Marks in LDS, for each token of tile [t0, t1), the sequence that starts or
// ends there (-1: none), and runs f(n) for the empty sequences in it.
template <typename F>
__device__ __forceinline__ void mark_tokens(const Chain &p, int chunk, int t0, int t1, int *s_start, int *s_end, F f) {
    for (int i = threadIdx.x; i < kTc; i += 256) s_start[i] = s_end[i] = -1;
    __syncthreads();
    for (int n = p.tab[chunk] + threadIdx.x; n <= p.N; n += 256) {
        const int v = p.cu[n];
        if (v > t1) break;
        if (n < p.N) {
            const bool empty = p.cu[n + 1] == v;
            if (empty && (v < t1 || t1 == p.T)) f(n);
            if (!empty && v < t1) s_start[v - t0] = n;
        }
        if (n > 0 && v > t0 && p.cu[n - 1] < v) s_end[v - 1 - t0] = n - 1;
    }
    __syncthreads();
}

template <typename x_t, typename l_t, typename h_t, int V, bool PACKED>
__device__ __forceinline__ void scan_fwd_tile(const Chain &p, int64_t chain, const x_t *__restrict__ x,
                                                       const l_t *__restrict__ la, const float *init, float *fin,
                                                       h_t *__restrict__ h) {
    constexpr int LPR = kCw / V, G = 256 / LPR, TT = kElems / V;
    static_assert(G * TT == kTc, "the threads' tokens fill the tile");
    __shared__ float sA[G][kCw], sH[G][kCw];
    __shared__ int s_start[PACKED ? kTc : 1], s_end[PACKED ? kTc : 1], s_k;
    const int k = draw_place(p, chain, &s_k);
    const int row = (int)quotient(chain, p.ntile), col0 = (int)(chain - (int64_t)row * p.ntile) * kCw;
    const int tid = threadIdx.x, lp = tid % LPR, g = tid / LPR;
    const int t0 = k * kTc, len = min(kTc, p.T - t0);
    const int ch = col0 + lp * V;
    const bool live = ch < p.D;                       // V divides D: all of a thread's channels or none
    const int cc = live ? ch : 0;
    const int64_t base = ((int64_t)row * p.T + t0) * p.D;

    x_t xr[TT][V];
    l_t lr[TT][V];
    if (len > 0) {
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const uint32_t off = (uint32_t)min(g * TT + i, len - 1) * (uint32_t)p.D + (uint32_t)cc;
            load_vec<l_t, V>(la + base + off, lr[i]);
            load_vec<x_t, V>(x + base + off, xr[i]);
        }
    }
    uint32_t starts = 0;
    if constexpr (PACKED) {
        mark_tokens(p, k, t0, t0 + len, s_start, s_end, [&](int n) {
            if (fin && fin != init)
                for (int c = col0; c < min(col0 + kCw, p.D); ++c)
                    fin[(int64_t)n * p.D + c] = init ? init[(int64_t)n * p.D + c] : 0.f;
        });
    }
    float a[TT][V], v[TT][V], A[V], H[V];
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = 1.f, H[j] = 0.f;
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        const bool in = g * TT + i < len;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            a[i][j] = in ? exp_gate(to_f32(lr[i][j])) : 1.f;
            v[i][j] = in ? to_f32(xr[i][j]) : 0.f;
        }
        if constexpr (PACKED) {
            const int n = s_start[g * TT + i];
            if (n >= 0) {
                starts |= 1u << i;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (init && live) v[i][j] = fmaf(a[i][j], init[(int64_t)n * p.D + ch + j], v[i][j]);
                    A[j] = -0.f;
                    H[j] = v[i][j];
                }
                continue;
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            H[j] = fmaf(a[i][j], H[j], v[i][j]);
            A[j] = PACKED && starts ? -0.f : A[j] * a[i][j];
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        sA[g][lp * V + j] = A[j];
        sH[g][lp * V + j] = H[j];
    }
    __syncthreads();
    if (tid < kCw) {                                  // one wave, a lane per channel of the tile
        float ga[G], gh[G], bA = 1.f, bH = 0.f;
#pragma unroll
        for (int q = 0; q < G; ++q) {
            ga[q] = sA[q][tid];
            gh[q] = sH[q][tid];
            bH = apply<PACKED>(ga[q], gh[q], bH);
            bA = PACKED && (forgets(ga[q]) || forgets(bA)) ? -0.f : bA * ga[q];
        }
        const bool on = col0 + tid < p.D;
        const int64_t sidx = (int64_t)row * p.D + col0 + tid;
        float s = chain_state<PACKED>(p, chain, k, tid, bA, bH, !PACKED && init && on ? init[sidx] : 0.f);
#pragma unroll
        for (int q = 0; q < G; ++q) {                 // the state that enters each thread group
            sH[q][tid] = s;
            s = apply<PACKED>(ga[q], gh[q], s);
        }
        if (!PACKED && fin && on && k + 1 >= p.nchunk) fin[sidx] = s;
    }
    __syncthreads();
    if (!live) return;
    float s[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = sH[g][lp * V + j];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        const int t = g * TT + i;
        if (t >= len) break;
        h_t o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float n = fmaf(a[i][j], s[j], v[i][j]);
            s[j] = PACKED && (starts >> i & 1) ? v[i][j] : n;
            o[j] = round_to<h_t>(s[j]);
        }
        store_vec<h_t, V>(h + base + ((uint32_t)t * (uint32_t)p.D + (uint32_t)ch), o);
        if constexpr (PACKED) {
            if (fin && s_end[t] >= 0)
#pragma unroll
                for (int j = 0; j < V; ++j) fin[(int64_t)s_end[t] * p.D + ch + j] = s[j];
        }
    }
}

template <typename x_t, typename l_t, typename h_t, int V, bool PACKED>
__global__ __launch_bounds__(256) void scan_fwd_kernel(Chain p, const x_t *__restrict__ x, const l_t *__restrict__ la,
                                                       const float *init, float *fin, h_t *__restrict__ h) {
    if (PACKED && p.meta[1] != 0) return;
    if (!PACKED && blockIdx.x == 0 && threadIdx.x == 0) p.meta[0] = p.meta[1] = 0;
    for (int64_t b = blockIdx.x; b < p.blocks; b += gridDim.x) {
        scan_fwd_tile<x_t, l_t, h_t, V, PACKED>(p, modulo(b, p.nchain), x, la, init, fin, h);
        __syncthreads();   // the tile's LDS is no longer read
    }
}

template <typename x_t, typename l_t, typename h_t, int V, bool PACKED>
__device__ __forceinline__ void scan_bwd_tile(const Chain &p, int64_t chain, const l_t *__restrict__ la,
                                                       const h_t *__restrict__ h, const float *__restrict__ init,
                                                       const h_t *__restrict__ dh, const float *__restrict__ dfin,
                                                       x_t *__restrict__ dx, l_t *__restrict__ dla,
                                                       float *__restrict__ dinit) {
    constexpr int LPR = kCw / V, G = 256 / LPR, TT = kElems / V;
    __shared__ float sA[G][kCw], sH[G][kCw];
    __shared__ int s_start[PACKED ? kTc : 1], s_end[PACKED ? kTc : 1], s_k;
    const int k = draw_place(p, chain, &s_k);
    const int chunk = p.nchunk > 0 ? p.nchunk - 1 - k : 0;   // the chain runs from the last tile to the first
    const int row = (int)quotient(chain, p.ntile), col0 = (int)(chain - (int64_t)row * p.ntile) * kCw;
    const int tid = threadIdx.x, lp = tid % LPR, g = tid / LPR;
    const int t0 = chunk * kTc, len = min(kTc, p.T - t0);
    const int ch = col0 + lp * V;
    const bool live = ch < p.D;
    const int cc = live ? ch : 0;
    const int64_t base = ((int64_t)row * p.T + t0) * p.D;

    h_t gr[TT][V], hr[TT][V];
    l_t lr[TT][V];
    if (len > 0) {
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const int t = min(g * TT + i, len - 1);
            const uint32_t off = (uint32_t)t * (uint32_t)p.D + (uint32_t)cc;
            load_vec<l_t, V>(la + base + off, lr[i]);
            load_vec<h_t, V>(dh + base + off, gr[i]);
            // h of the token before; at the very first token of a row it is not used
            load_vec<h_t, V>(h + base + (t0 + t > 0 ? (int64_t)off - p.D : (int64_t)off), hr[i]);
        }
    }
    uint32_t ends = 0;
    if constexpr (PACKED) {
        mark_tokens(p, chunk, t0, t0 + len, s_start, s_end, [&](int n) {
            if (dinit)
                for (int c = col0; c < min(col0 + kCw, p.D); ++c)
                    dinit[(int64_t)n * p.D + c] = dfin ? dfin[(int64_t)n * p.D + c] : 0.f;
        });
    }
    float a[TT][V], v[TT][V], A[V], H[V];
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = 1.f, H[j] = 0.f;
#pragma unroll
    for (int i = TT - 1; i >= 0; --i) {
        const bool in = g * TT + i < len;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            a[i][j] = in ? exp_gate(to_f32(lr[i][j])) : 1.f;
            v[i][j] = in ? to_f32(gr[i][j]) : 0.f;
        }
        if constexpr (PACKED) {
            const int n = s_end[g * TT + i];
            if (n >= 0) {
                ends |= 1u << i;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (dfin && live) v[i][j] += dfin[(int64_t)n * p.D + ch + j];
                    A[j] = -0.f;
                    H[j] = a[i][j] * v[i][j];
                }
                continue;
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            H[j] = a[i][j] * (v[i][j] + H[j]);
            A[j] = PACKED && ends ? -0.f : A[j] * a[i][j];
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        sA[g][lp * V + j] = A[j];
        sH[g][lp * V + j] = H[j];
    }
    __syncthreads();
    if (tid < kCw) {
        float ga[G], gh[G], bA = 1.f, bH = 0.f;
#pragma unroll
        for (int q = G - 1; q >= 0; --q) {
            ga[q] = sA[q][tid];
            gh[q] = sH[q][tid];
            bH = apply<PACKED>(ga[q], gh[q], bH);
            bA = PACKED && (forgets(ga[q]) || forgets(bA)) ? -0.f : bA * ga[q];
        }
        const bool on = col0 + tid < p.D;
        const int64_t sidx = (int64_t)row * p.D + col0 + tid;
        float s = chain_state<PACKED>(p, chain, k, tid, bA, bH, !PACKED && dfin && on ? dfin[sidx] : 0.f);
#pragma unroll
        for (int q = G - 1; q >= 0; --q) {
            sH[q][tid] = s;
            s = apply<PACKED>(ga[q], gh[q], s);
        }
        if (!PACKED && dinit && on && chunk == 0) dinit[sidx] = s;
    }
    __syncthreads();
    if (!live) return;
    float e[V];
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = sH[g][lp * V + j];
#pragma unroll
    for (int i = TT - 1; i >= 0; --i) {
        const int t = g * TT + i;
        if (t >= len) continue;
        int n = -1;
        bool begin = !PACKED && t0 + t == 0;
        if constexpr (PACKED) {
            n = s_start[t];
            begin = n >= 0;
        }
        x_t ox[V];
        l_t ol[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float q = PACKED && (ends >> i & 1) ? v[i][j] : v[i][j] + e[j];
            e[j] = a[i][j] * q;
            float past = to_f32(hr[i][j]);
            if (begin) past = init ? init[(int64_t)(PACKED ? n : row) * p.D + ch + j] : 0.f;
            ox[j] = round_to<x_t>(q);
            ol[j] = round_to<l_t>(e[j] * past);
        }
        const uint32_t off = (uint32_t)t * (uint32_t)p.D + (uint32_t)ch;
        store_vec<x_t, V>(dx + base + off, ox);
        store_vec<l_t, V>(dla + base + off, ol);
        if constexpr (PACKED) {
            if (dinit && begin)
#pragma unroll
                for (int j = 0; j < V; ++j) dinit[(int64_t)n * p.D + ch + j] = e[j];
        }
    }
}

template <typename x_t, typename l_t, typename h_t, int V, bool PACKED>
__global__ __launch_bounds__(256) void scan_bwd_kernel(Chain p, const l_t *__restrict__ la,
                                                       const h_t *__restrict__ h, const float *__restrict__ init,
                                                       const h_t *__restrict__ dh, const float *__restrict__ dfin,
                                                       x_t *__restrict__ dx, l_t *__restrict__ dla,
                                                       float *__restrict__ dinit) {
    if (PACKED && p.meta[1] != 0) return;
    if (!PACKED && blockIdx.x == 0 && threadIdx.x == 0) p.meta[0] = p.meta[1] = 0;
    for (int64_t b = blockIdx.x; b < p.blocks; b += gridDim.x) {
        scan_bwd_tile<x_t, l_t, h_t, V, PACKED>(p, modulo(b, p.nchain), la, h, init, dh, dfin, dx, dla, dinit);
        __syncthreads();   // the tile's LDS is no longer read
    }
}

// Fills `c` and enqueues the setup kernel where the call needs one.
static hipError_t scan_setup(const ScanArgs &a, Chain &c, hipStream_t st) {
    const bool packed = a.cu_seqlens != nullptr;
    const auto w = scan_workspace_layout(a.B, a.T, a.D, a.N, packed);
    char *ws = static_cast<char *>(a.workspace);
    c.T = a.T, c.D = a.D, c.N = a.N, c.nchunk = (int)w.chunks, c.ntile = (int)w.tiles;
    c.cu = a.cu_seqlens;
    c.meta = reinterpret_cast<int32_t *>(ws);
    c.tab = reinterpret_cast<int32_t *>(ws + w.off_tab);
    c.ctr = reinterpret_cast<int32_t *>(ws + w.off_ctr);
    c.agg = reinterpret_cast<uint64_t *>(ws + w.off_agg);
    c.pre = reinterpret_cast<uint64_t *>(ws + w.off_pre);
    c.nchain = w.rows * w.tiles;
    c.blocks = (w.chunks > 0 ? w.chunks : 1) * c.nchain;
    if (w.chunks <= 1 && !packed) return hipSuccess;
    const int64_t words16 = (int64_t)(w.total - w.off_agg) / 16;
    int64_t blocks = (words16 / 4 + 255) / 256;
    blocks = blocks < 1 ? 1 : (blocks > 2048 ? 2048 : blocks);
    ProfScope prof("gdn_scan_setup", st);
    // an empty packed batch still has one tile: it hands on the states
    scan_setup_kernel<<<(unsigned)blocks, 256, 0, st>>>(a.N, a.T, w.chunks > 0 ? (int)w.chunks : 1, a.cu_seqlens,
                                                        c.meta, reinterpret_cast<int32_t *>(ws + w.off_tab), c.ctr,
                                                        w.chunks > 1 ? c.nchain : 0,
                                                        reinterpret_cast<u32x4_t *>(ws + w.off_agg), words16);
    return hipGetLastError();
}

// Loads of 4 channels where every row starts on one (D a multiple of 4), of
// one otherwise.
template <typename F>
static hipError_t with_shape(const ScanArgs &a, F f) {
    using std::integral_constant;
    const bool packed = a.cu_seqlens != nullptr;
    auto vec = [&](auto v) {
        return packed ? f(v, integral_constant<bool, true>{}) : f(v, integral_constant<bool, false>{});
    };
    return a.D % 4 == 0 ? vec(integral_constant<int, 4>{}) : vec(integral_constant<int, 1>{});
}

hipError_t launch_scan_fwd(const ScanArgs &a, hipStream_t st) {
    Chain c;
    hipError_t e = scan_setup(a, c, st);
    if (e != hipSuccess) return e;
    const unsigned blocks = (unsigned)(c.blocks < kMaxBlocks ? c.blocks : kMaxBlocks);
    ProfScope prof("gdn_scan_fwd", st);
    return with_types(a.in_dtype, a.gate_dtype, a.out_dtype, [&](auto x, auto l, auto h) {
        return with_shape(a, [&](auto v, auto packed) {
            using x_t = decltype(x);
            using l_t = decltype(l);
            using h_t = decltype(h);
            scan_fwd_kernel<x_t, l_t, h_t, decltype(v)::value, decltype(packed)::value>
                <<<blocks, 256, 0, st>>>(c, static_cast<const x_t *>(a.x),
                                                   static_cast<const l_t *>(a.log_alpha), a.init_state, a.final_state,
                                                   static_cast<h_t *>(a.h));
            return hipGetLastError();
        });
    });
}

hipError_t launch_scan_bwd(const ScanArgs &a, hipStream_t st) {
    Chain c;
    hipError_t e = scan_setup(a, c, st);
    if (e != hipSuccess) return e;
    const unsigned blocks = (unsigned)(c.blocks < kMaxBlocks ? c.blocks : kMaxBlocks);
    ProfScope prof("gdn_scan_bwd", st);
    return with_types(a.in_dtype, a.gate_dtype, a.out_dtype, [&](auto x, auto l, auto h) {
        return with_shape(a, [&](auto v, auto packed) {
            using x_t = decltype(x);
            using l_t = decltype(l);
            using h_t = decltype(h);
            scan_bwd_kernel<x_t, l_t, h_t, decltype(v)::value, decltype(packed)::value>
                <<<blocks, 256, 0, st>>>(c, static_cast<const l_t *>(a.log_alpha),
                                                   static_cast<const h_t *>(a.h), a.init_state,
                                                   static_cast<const h_t *>(a.d_h), a.d_final,
                                                   static_cast<x_t *>(a.dx), static_cast<l_t *>(a.dlog_alpha),
                                                   a.d_init);
            return hipGetLastError();
        });
    });
}

// ---- single step -----------------------------------------------------------------

template <typename x_t, typename l_t, typename h_t>
__global__ __launch_bounds__(256) void scan_step_kernel(int64_t n, float *__restrict__ state,
                                                        const x_t *__restrict__ x, const l_t *__restrict__ la,
                                                        h_t *__restrict__ h) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const float s = fmaf(exp_gate(to_f32(la[i])), state[i], to_f32(x[i]));
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
