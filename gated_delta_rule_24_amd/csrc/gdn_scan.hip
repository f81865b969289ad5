// Gated linear recurrence h_t = alpha_t h_{t-1} + x_t per channel, its
// gradient and its single step.  All three are bound by HBM: no value is used
// twice, and a token costs one exp and two or three multiply-adds a channel.
//
// Sequences in one pass: a form of the published single-pass scan with
// look-back.  Tokens compose as affine maps h -> A h + H:
//   (A1, H1) then (A2, H2)  =  (A1 A2, A2 H1 + H2).
// A block takes a tile of 128 tokens x 128 channels, reads it once into
// registers, forms its threads' maps, joins them in LDS, gets the state that
// enters the tile, runs the recurrence from the registers and writes the
// result: every tensor crosses HBM once, whatever the length.  The state that
// enters a tile comes from the tiles before it in the same chain (batch row
// and channel tile).  A chain's tiles form groups of kGroup, its groups
// sections of kGroup:
//   - a tile publishes its own map (agg) as soon as it has it;
//   - the last tile of a group publishes the group's map (grp), the last of a
//     section the state that leaves it (pre);
//   - a tile joins the maps of the groups before its own in the section and
//     of the tiles before it in the group, in order, and applies them to the
//     state that entered the section.
// The order of every sum is fixed, so equal calls give equal bits, and only
// one hand-over per 64 tiles is serial.
// Every published value is one 8-byte word, written and read by relaxed
// device-scope atomics, so a word is whole or not there: scan_setup_kernel
// fills the words with kEmpty, which no published word equals (a not-a-number H
// is published in one form).  No fence is needed, as nothing but the word
// itself is handed over.
// Every wait ends, in whatever order the blocks run: tiles are given to blocks
// in the order of their chain, so the tiles before a block's own have as a
// rule begun before it; but a block that has looked `patience` times for
// words (about 4 ms) waits no longer and works out the maps of all tiles before
// its own itself, in the same order of sums.
//
// Measured (MI355X, a large copy reaches 5.4 TB/s): 4 x 4096 x 2048 from bf16
// with fp32 gates 54 us (5.0 TB/s), its gradient 91 us (5.2), 32768 x 4096 in
// fp16 backward 249 us (5.4), 50408 packed tokens x 2048 in bf16 136 us (4.6),
// their gradient 204 us (5.1), with fp32 gates and h 337 us (5.5).  The form of
// the tile is the same whatever the sizes: few tiles or few channels leave most
// of the GPU idle (3 x 1001 x 333 in fp32 13 us, 65536 x 16 in bf16 17 us, where a
// copy of their bytes takes 2 and 1).
// Tiles are 256 bytes a row because a plain copy in tiles of 128 tokens runs at
// 4.9 TB/s with rows of 128 bytes, 5.5 with 256, 6.0 with 512; 256 channels in
// blocks of 512 threads leave 64 tokens a tile and twice the words (prefill 59
// us).  Loads and stores that pass the caches by save 7%.  What is left is a
// block's life: one load latency and one or two hand-overs per tile with three
// (16-bit operands) or two blocks a CU to cover them.  Drawing a tile's place
// from a counter instead costs 2-7%; keeping blocks on their CUs with the next
// tile's loads in flight leaves the words too late (75 us for prefill).
//
// The gradient is the same recurrence backwards in e_t = alpha_t g_t,
//   g_t = dh_t + e_{t+1},  e_t = alpha_t g_t,
// with dx_t = g_t, dlog_alpha_t = e_t h_{t-1}.
//
// Packed batches are one chain over all tokens, cut at sequence starts: a map
// that crosses a start forgets what enters it.  Such a map has kForgets for A
// (no product of exponentials is negative), and forgetting is a selection, not
// a product with zero, so not-a-number and infinite states stay in their own
// sequence.  Inside a sequence an infinite state stays infinite: products of
// decays do not fall to 0 by underflow (times).
#include "gdn_device.h"
#include "gdn_ops.h"
#include "gdn_types.h"

#include <stdlib.h>

#include <algorithm>

// Products and sums are fused only where fmaf says so: the same recurrence is
// written in unrolled and in plain loops, whose bits have to agree.
#pragma clang fp contract(off)

namespace gdn {

constexpr int kCw = 128;        // channels of a tile
constexpr int kNt = 512;        // threads of a block
constexpr int kElems = 32;      // elements per thread
constexpr int kTc = kNt * kElems / kCw;   // tokens of a tile: 128
constexpr int kGroup = 8;       // tiles per group of a chain, and groups per section
constexpr int kShortRow = 32;   // tokens of a row that a thread takes alone
constexpr uint64_t kEmpty = ~0ull;
constexpr int64_t kMaxGridX = 1 << 20;
constexpr int kPatience = 4096; // looks at a word before a block helps itself

static int64_t scan_tiles(int64_t n, int64_t w) { return (n + w - 1) / w; }

// Whether final states over the initial ones make the kernels read a copy:
// initial states are read by more than one block, or twice, and the sequence
// may have ended in another block by then.  Only single tiles of whole vectors
// are safe.
static bool keeps_init(bool packed, int32_t D, int64_t chunks) { return packed || D % 4 != 0 || chunks > 1; }

ScanWorkspace scan_workspace_layout(int32_t B, int32_t T, int32_t D, int32_t N, bool packed) {
    ScanWorkspace w;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    w.rows = packed ? 1 : B;
    w.chunks = scan_tiles(T, kTc);
    w.tiles = scan_tiles(D, kCw);
    const bool chained = w.chunks > 1;
    const int64_t words = chained ? w.rows * w.tiles * kCw : 0;
    size_t at = 256;                                   // meta
    w.off_seq = at;
    at += packed ? up((size_t)T * 4) : 0;
    w.off_init = at;
    at += keeps_init(packed, D, w.chunks) ? up((size_t)N * D * 4) : 0;
    w.off_agg = at;
    at += up((size_t)words * w.chunks * 8);
    w.off_grp = at;
    at += up((size_t)words * scan_tiles(w.chunks, kGroup) * 8);
    w.off_pre = at;
    at += up((size_t)words * scan_tiles(w.chunks, kGroup * kGroup) * 8);
    w.total = at;
    return w;
}

// Empties the words; packed: checks cu_seqlens (codes as in
// chunk_table_kernel) and writes down each token's sequence; copies the initial
// states where need be (keeps_init).
__global__ __launch_bounds__(256) void scan_setup_kernel(int N, int T, const int32_t *__restrict__ cu,
                                                         int32_t *__restrict__ meta, int32_t *__restrict__ seq,
                                                         u32x4_t *__restrict__ words, int64_t nwords16,
                                                         const float *__restrict__ init, float *__restrict__ keep,
                                                         int64_t nkeep) {
    const int64_t tid = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)gridDim.x * 256;
    for (int64_t i = tid; i < nwords16; i += all) words[i] = u32x4_t{~0u, ~0u, ~0u, ~0u};
    for (int64_t i = tid; i < nkeep; i += all) keep[i] = init[i];
    if (!cu) return;
    for (int64_t t = tid; t < T; t += all) {
        int lo = 1, hi = N;            // the first n >= 1 with cu[n] > t (N if there is none)
        while (lo < hi) {
            const int mid = lo + ((hi - lo) >> 1);
            if (cu[mid] <= t) lo = mid + 1;
            else hi = mid;
        }
        seq[t] = lo - 1;
    }
    if (blockIdx.x == 0) {
        __shared__ int s_code;
        if (threadIdx.x == 0) s_code = 0;
        __syncthreads();
        int code = 0;
        for (int64_t n = threadIdx.x; n <= N; n += 256) {
            const int v = cu[n];
            if (n == 0 && v != 0) code |= 1;
            if (n > 0 && cu[n - 1] > v) code |= 2;
            if (n == N && v != T) code |= 4;
        }
        if (code) atomicOr(&s_code, code);
        __syncthreads();
        if (threadIdx.x == 0) {
            meta[0] = T;
            meta[1] = (s_code & 1) ? 1 : ((s_code & 2) ? 2 : (s_code ? 3 : 0));
        }
    }
}

// ---- maps ---------------------------------------------------------------------

// A of a map that forgets: all bits set.  A not-a-number with its sign set counts
// as that too, which changes nothing: the map's H is not-a-number as well.
#define kForgets __uint_as_float(~0u)
__device__ __forceinline__ bool forgets(float A) { return (int32_t)__float_as_uint(A) < 0; }
// What map (A, H) makes of state s.
template <bool PACKED>
__device__ __forceinline__ float apply(float A, float H, float s) {
    const float v = fmaf(A, s, H);
    return PACKED && forgets(A) ? H : v;
}
// A product of decays is 0 only if a decay is: underflow stops at the smallest
// number, 2^-149, so that an infinite state that decays stays infinite, as it
// does token by token.  A finite state is off by at most 2^-149 of itself, a step
// of the product's type there.  Decays are not negative, so their bits are
// ordered as they are, not-a-number on top and what forgets above all.  A chain
// of 512 tiles pays 0.3 to 0.8 us for it (65536 x 16, 17 us), other calls less
// than 1%.
__device__ __forceinline__ float above_zero(float product, bool none_is_zero) {
    return __uint_as_float(max(__float_as_uint(product), none_is_zero ? 1u : 0u));
}
template <bool PACKED>
__device__ __forceinline__ float times(float A, float nA) {
    const uint32_t a = __float_as_uint(A), n = __float_as_uint(nA);
    const uint32_t least = min(min(a, n), 1u), forget = PACKED ? (uint32_t)((int32_t)(a | n) >> 31) : 0u;
    return __uint_as_float(max(max(__float_as_uint(A * nA), least), forget));
}
// (A, H) followed by (nA, nH).
template <bool PACKED>
__device__ __forceinline__ void join(float &A, float &H, float nA, float nH) {
    H = apply<PACKED>(nA, nH, H);
    A = times<PACKED>(A, nA);
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
// exp(x): exp2's instruction on x log2(e).  It gives 0 below 2^-126, which is off
// by at most 2^-126 of a finite state.
__device__ __forceinline__ float exp_gate(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
// the same on any element's address (rows of D elements start anywhere)
typedef u32x2_t loose2_t __attribute__((aligned(2)));
typedef u32x4_t loose4_t __attribute__((aligned(2)));
// Every element is used once: loads and stores that leave no trace in the
// caches.  The loose types are named at each access: a template argument would
// lose their alignment, and the compiler would take addresses for aligned that
// are not.
__device__ __forceinline__ void stream_load(const char *p, uint16_t &r) {
    r = __builtin_nontemporal_load(reinterpret_cast<const uint16_t *>(p));
}
__device__ __forceinline__ void stream_load(const char *p, uint32_t &r) {   // an fp32 element
    r = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(p));
}
__device__ __forceinline__ void stream_load(const char *p, u32x2_t &r) {
    r = __builtin_nontemporal_load(reinterpret_cast<const loose2_t *>(p));
}
__device__ __forceinline__ void stream_load(const char *p, u32x4_t &r) {
    r = __builtin_nontemporal_load(reinterpret_cast<const loose4_t *>(p));
}
__device__ __forceinline__ void stream_store(char *p, uint16_t r) {
    __builtin_nontemporal_store(r, reinterpret_cast<uint16_t *>(p));
}
__device__ __forceinline__ void stream_store(char *p, uint32_t r) {
    __builtin_nontemporal_store(r, reinterpret_cast<uint32_t *>(p));
}
__device__ __forceinline__ void stream_store(char *p, u32x2_t r) {
    __builtin_nontemporal_store(r, reinterpret_cast<loose2_t *>(p));
}
__device__ __forceinline__ void stream_store(char *p, u32x4_t r) {
    __builtin_nontemporal_store(r, reinterpret_cast<loose4_t *>(p));
}
// The registers that hold B bytes of consecutive elements.
template <int B>
using words_t = std::conditional_t<
    B == 2, uint16_t, std::conditional_t<B == 4, uint32_t, std::conditional_t<B == 8, u32x2_t, u32x4_t>>>;

// V consecutive elements as loaded (16-bit types two to a register).  Values
// are converted each time they are used: the registers that this saves let
// one block more share a CU.
template <typename T, int V>
struct Held {
    static constexpr int W = (V * (int)sizeof(T) + 3) / 4;
    uint32_t w[W];
    // element `off` of a uniform base (32-bit byte offsets: one scalar base for all of a thread's loads)
    __device__ __forceinline__ void load(const T *base, uint32_t off) {
        const char *p = reinterpret_cast<const char *>(base) + (uint32_t)(off * (uint32_t)sizeof(T));
        words_t<V * (int)sizeof(T)> r;
        stream_load(p, r);
        if constexpr (W == 1)
            w[0] = r;
        else
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = r[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    // The registers as a new value: what was computed from them before is not kept for later.
    __device__ __forceinline__ void touch() {
#pragma unroll
        for (int i = 0; i < W; ++i) asm volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (std::is_same_v<T, float>)
            return __uint_as_float(w[j]);
        else if constexpr (std::is_same_v<T, bf16_t>)
            return __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
        else
            return (float)__builtin_bit_cast(_Float16, (uint16_t)(j & 1 ? w[j / 2] >> 16 : w[j / 2]));
    }
    __device__ __forceinline__ void set(int j, float v) {   // fp32 only
        w[j] = __float_as_uint(v);
    }
};
// A gate: log alpha as loaded; alpha itself takes the place of an fp32 one.
template <typename T, int V>
struct Gate : Held<T, V> {
    __device__ __forceinline__ float first(int j) {
        const float a = exp_gate(this->get(j));
        if constexpr (std::is_same_v<T, float>) this->set(j, a);
        return a;
    }
    __device__ __forceinline__ float again(int j) const {
        if constexpr (std::is_same_v<T, float>) return this->get(j);
        return exp_gate(this->get(j));
    }
};
// The products A of a thread's decays where some came out as 0 (above_zero).
// Whether a decay is 0 is seen from the gates as they are held, which takes no
// registers beside theirs: fp32 decays, or the bits of 16-bit log alpha, whose
// decay is 0 from kZeroDecay on.  Taking `times` for every token instead costs
// 1-2% in packed calls and with fp32 gates.
template <typename T>
constexpr uint32_t kZeroDecay = std::is_same_v<T, bf16_t> ? 0xC2AFu : 0xD576u;   // -87.5, -87.375
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
template <typename T, int V, int TT>
__device__ __forceinline__ void mend_products(float (&A)[V], const Gate<T, V> (&gate)[TT]) {
    bool zero = false;
#pragma unroll
    for (int j = 0; j < V; ++j) zero |= A[j] == 0.f;
    if (!zero) return;
    constexpr int W = Gate<T, V>::W;
#pragma unroll
    for (int k = 0; k < W; ++k) {
        if constexpr (std::is_same_v<T, float>) {
            uint32_t least = 1;
#pragma unroll
            for (int i = 0; i < TT; ++i) least = min(least, gate[i].w[k]);
            A[k] = above_zero(A[k], least != 0);
        } else {
            u16x2_t most = 0;
#pragma unroll
            for (int i = 0; i < TT; ++i)
                most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2_t, gate[i].w[k]));
            A[2 * k] = above_zero(A[2 * k], most[0] < kZeroDecay<T>);
            if constexpr (V > 1) A[2 * k + 1] = above_zero(A[2 * k + 1], most[1] < kZeroDecay<T>);
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *base, uint32_t off, const T (&v)[V]) {
    char *p = reinterpret_cast<char *>(base) + (uint32_t)(off * (uint32_t)sizeof(T));
    struct A {
        T e[V];
    } a;
#pragma unroll
    for (int j = 0; j < V; ++j) a.e[j] = v[j];
    stream_store(p, __builtin_bit_cast(words_t<(int)sizeof(A)>, a));
}

// ---- the chain --------------------------------------------------------------------

struct Chain {
    int T, D, N, nchunk, ntile;
    int64_t nchain, blocks;        // chains, tiles of all chains
    const int32_t *cu;
    int32_t *meta;
    const int32_t *seq;
    int patience;
    uint64_t *agg, *grp, *pre;
};

// The state entering tile `k` (its place in the chain) for column `c`, from
// the tile's own map (A, H).  Publishes what the tiles after it need and waits
// for the tiles before it; where a word does not come, map(j, A, H) works out
// the map of tile j.  `first` is the state that enters the chain.
template <bool PACKED, typename F>
__device__ __forceinline__ float chain_state(const Chain &p, int64_t chain, int k, int c, float A, float H,
                                             float first, F map) {
    if (p.nchunk <= 1) return first;
    constexpr int kG = kGroup;
    const int s = k % kG, r = k / kG % kG, R = k / (kG * kG);
    uint64_t *agg = p.agg + (chain * p.nchunk + (k - s)) * kCw + c;
    uint64_t *grp = p.grp + (chain * ((p.nchunk + kG - 1) / kG) + R * kG) * kCw + c;
    uint64_t *pre = p.pre + (chain * ((p.nchunk + kG * kG - 1) / (kG * kG)) + R) * kCw + c;
    const bool more = k + 1 < p.nchunk;
    if (more && s < kG - 1) put(agg + s * kCw, word(A, H));
    int looks = 0;
    bool late = false;
    auto wait = [&](uint64_t &v, const uint64_t *at) {
        while (!late && __any(v == kEmpty)) {
            if (++looks > p.patience) {
                late = true;
                break;
            }
            __builtin_amdgcn_s_sleep(2);
            v = get(at);
        }
    };
    auto upper = [](uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); };
    auto lower = [](uint64_t v) { return __uint_as_float((uint32_t)v); };
    // Look at the words of a kind once, then wait for each that is not there
    // yet.
    auto join_words = [&](float &mA, float &mH, const uint64_t *at, int n) {
        uint64_t w[kG - 1];
#pragma unroll
        for (int j = 0; j < kG - 1; ++j) w[j] = j < n ? get(at + j * kCw) : 0;
#pragma unroll
        for (int j = 0; j < kG - 1; ++j)
            if (j < n) {
                wait(w[j], at + j * kCw);
                join<PACKED>(mA, mH, upper(w[j]), lower(w[j]));
            }
    };
    // joined: the tiles before this one in its group, the groups before that
    // in its section; in: the state that enters the section
    float gA = 1.f, gH = 0.f, sA = 1.f, sH = 0.f, in = first;
    auto publish_group = [&] {
        float lA = gA, lH = gH;
        join<PACKED>(lA, lH, A, H);
        if (more && s == kG - 1 && r < kG - 1) put(grp + r * kCw, word(lA, lH));
    };
    join_words(gA, gH, agg, s);
    if (!late) {
        publish_group();
        join_words(sA, sH, grp, r);
        if (R > 0) {
            uint64_t u = get(pre);
            wait(u, pre);
            in = lower(u);
        }
    }
    if (late) {
        gA = sA = 1.f, gH = sH = 0.f, in = first;
        for (int j = 0; j < k; ++j) {
            float tA, tH, eA = sA, eH = sH;
            map(j, tA, tH);
            join<PACKED>(eA, eH, gA, gH);
            const float out = apply<PACKED>(tA, tH, apply<PACKED>(eA, eH, in));
            join<PACKED>(gA, gH, tA, tH);
            if (j % kG == kG - 1) {
                if (j / kG % kG == kG - 1) {
                    in = out;
                    sA = 1.f, sH = 0.f;
                } else {
                    join<PACKED>(sA, sH, gA, gH);
                }
                gA = 1.f, gH = 0.f;
            }
        }
        publish_group();
    }
    join<PACKED>(sA, sH, gA, gH);
    in = apply<PACKED>(sA, sH, in);
    if (more && s == kG - 1 && r == kG - 1) put(pre + kCw, word(0.f, apply<PACKED>(A, H, in)));
    return in;
}

// Whole-number division, in 32 bits where that is enough.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// This block's chain and its place there; false past the last tile.
__device__ __forceinline__ bool take_tile(const Chain &p, int64_t &chain, int &k) {
    const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (b >= p.blocks) return false;
    k = (int)quotient(b, p.nchain);
    chain = b - k * p.nchain;
    return true;
}

// Waves per SIMD that a kernel's registers should leave room for.  A thread's
// operands take kElems / 4 times (registers for 4 values) each; with three
// blocks a CU instead of two, packed 16-bit calls take 135 us instead of 145.
template <int V, typename... T>
constexpr int min_waves() {
    const int held = kElems / V * (... + Held<T, V>::W);
    return held <= 32 ? 6 : 4;
}

// Bit i: token t0 + i of the thread's TT tokens is the first (last) of its
// sequence.  s_seq[i]: the sequence of token i - 1 of the tile, -1 outside.
template <int TT>
__device__ __forceinline__ void edges(const int *s_seq, int t0, int len, uint32_t &starts, uint32_t &ends) {
    starts = ends = 0;
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        const int q = s_seq[t0 + i + 1];
        if (t0 + i < len) {
            starts |= q != s_seq[t0 + i] ? 1u << i : 0u;
            ends |= q != s_seq[t0 + i + 2] ? 1u << i : 0u;
        }
    }
}
// Loads what s_seq gets from this thread: token t0 - 1 + tid.
__device__ __forceinline__ int load_seq(const Chain &p, int t0) {
    const int64_t t = (int64_t)t0 - 1 + threadIdx.x;
    return threadIdx.x < kTc + 2 && t >= 0 && t < p.T ? p.seq[t] : -1;
}
// What empty sequences end with (begin with, for the gradient) is what they
// were given.  Rows of [N, D] are shared out over the blocks.
__device__ __forceinline__ void hand_on(const Chain &p, const float *from, float *to) {
    if (!to || to == from) return;
    for (int64_t n = (int64_t)blockIdx.y * gridDim.x + blockIdx.x; n < p.N; n += (int64_t)gridDim.x * gridDim.y)
        if (p.cu[n] == p.cu[n + 1])
            for (int c = threadIdx.x; c < p.D; c += kNt) to[n * p.D + c] = from ? from[n * p.D + c] : 0.f;
}

template <typename x_t, typename l_t, typename h_t, int V, bool PACKED>
__device__ __forceinline__ void scan_fwd_tile(const Chain &p, int64_t chain, int k, const x_t *__restrict__ x,
                                              const l_t *__restrict__ la, const float *init, float *fin,
                                              h_t *__restrict__ h) {
    constexpr int LPR = kCw / V, G = kNt / LPR, TT = kElems / V;
    static_assert(G * TT == kTc, "the threads' tokens fill the tile");
    static_assert(kNt >= kTc + 2, "one thread per entry of s_seq");
    __shared__ float sA[G][kCw], sH[G][kCw];
    __shared__ int s_seq[PACKED ? kTc + 2 : 1];
    const int row = (int)quotient(chain, p.ntile), col0 = (int)(chain - (int64_t)row * p.ntile) * kCw;
    const int tid = threadIdx.x, lp = tid % LPR, g = tid / LPR;
    const int t0 = k * kTc, len = min(kTc, p.T - t0);
    // a row's last thread ends with the row: the channels that it shares with
    // the thread before it are computed and written twice, with the same bits
    const bool live = col0 + lp * V < p.D;
    const int ch = min(col0 + lp * V, p.D - V);
    const int64_t base = ((int64_t)row * p.T + t0) * p.D;

    const int seq = PACKED ? load_seq(p, t0) : 0;
    Held<x_t, V> xr[TT];
    Gate<l_t, V> lr[TT];
    if (len > 0) {
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const uint32_t off = (uint32_t)min(g * TT + i, len - 1) * (uint32_t)p.D + (uint32_t)ch;
            lr[i].load(la + base, off);
            xr[i].load(x + base, off);
        }
    }
    // the state that enters the chain, for one channel of the tile
    const int wcol = col0 + tid / V * V;
    const int64_t wch = (int64_t)row * p.D + min(wcol, p.D - V) + tid % V;
    float edge = !PACKED && init && tid < kCw && wcol < p.D ? init[wch] : 0.f;
    uint32_t starts = 0, ends = 0;
    if constexpr (PACKED) {
        if (tid < kTc + 2) s_seq[tid] = seq;
        __syncthreads();
        edges<TT>(s_seq, g * TT, len, starts, ends);
    }
    if (len < kTc) {                                  // tokens past the end change nothing
#pragma unroll
        for (int i = 0; i < TT; ++i)
            if (g * TT + i >= len) {
                lr[i].zero();
                xr[i].zero();
            }
    }
    // before a sequence's first token the state is its initial one
    auto enter = [&](int i, float (&s)[V]) {
        if constexpr (PACKED)
            if (starts >> i & 1) {
                const int64_t n = s_seq[g * TT + i + 1];
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] = init && live ? init[n * p.D + ch + j] : 0.f;
            }
    };
    float A[V], H[V];
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = 1.f, H[j] = 0.f;
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        enter(i, H);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float a = lr[i].first(j);
            H[j] = fmaf(a, H[j], xr[i].get(j));
            A[j] *= a;
        }
    }
    mend_products(A, lr);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        sA[g][lp * V + j] = PACKED && starts ? kForgets : A[j];
        sH[g][lp * V + j] = H[j];
    }
    // The final state may go where the initial one is: it is here before
    // anything is published or written.
    asm volatile("" : "+v"(edge));
    __syncthreads();
    if (tid < kCw) {                                  // the first waves, a lane per channel of the tile
        float bA = 1.f, bH = 0.f;
#pragma unroll
        for (int q = 0; q < G; ++q) join<PACKED>(bA, bH, sA[q][tid], sH[q][tid]);
        // a tile before this one, token by token
        auto map = [&](int tile, float &tA, float &tH) {
            const int64_t at = (int64_t)row * p.T + (int64_t)tile * kTc;
            const int c = (int)(wch - (int64_t)row * p.D);
            tA = 1.f, tH = 0.f;
#pragma nounroll
            for (int q = 0; q < G; ++q) {
                float mA = 1.f, mH = 0.f;
                bool forget = false, nonzero = true;
#pragma nounroll
                for (int64_t t = at + q * TT; t < at + (q + 1) * TT; ++t) {
                    if (PACKED && (t == 0 || p.seq[t - 1] != p.seq[t])) {
                        mH = init ? init[(int64_t)p.seq[t] * p.D + c] : 0.f;
                        forget = true;
                    }
                    const float a = exp_gate(to_f32(la[t * p.D + c]));
                    mH = fmaf(a, mH, to_f32(x[t * p.D + c]));
                    mA *= a;
                    nonzero &= a != 0.f;
                }
                join<PACKED>(tA, tH, PACKED && forget ? kForgets : above_zero(mA, nonzero), mH);
            }
        };
        float s = chain_state<PACKED>(p, chain, k, tid, bA, bH, edge, map);
#pragma unroll
        for (int q = 0; q < G; ++q) {                 // the state that enters each thread group
            const float H = sH[q][tid];
            sH[q][tid] = s;
            s = apply<PACKED>(sA[q][tid], H, s);
        }
        if (!PACKED && fin && wcol < p.D && k + 1 >= p.nchunk) fin[wch] = s;
    }
    __syncthreads();
    if (!live) return;
    float s[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = sH[g][lp * V + j];
#pragma unroll
    for (int i = 0; i < TT; ++i) lr[i].touch(), xr[i].touch();
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        const int t = g * TT + i;
        if (t >= len) break;
        enter(i, s);
        h_t o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s[j] = fmaf(lr[i].again(j), s[j], xr[i].get(j));
            o[j] = round_to<h_t>(s[j]);
        }
        store_vec<h_t, V>(h + base, (uint32_t)t * (uint32_t)p.D + (uint32_t)ch, o);
        if constexpr (PACKED)
            if (fin && (ends >> i & 1))
#pragma unroll
                for (int j = 0; j < V; ++j) fin[(int64_t)s_seq[t + 1] * p.D + ch + j] = s[j];
    }
}

template <typename x_t, typename l_t, typename h_t, int V, bool PACKED>
__global__ __launch_bounds__(kNt, (min_waves<V, x_t, l_t>())) void scan_fwd_kernel(Chain p, const x_t *__restrict__ x,
                                                               const l_t *__restrict__ la, const float *init,
                                                               float *fin, h_t *__restrict__ h) {
    if (PACKED && p.meta[1] != 0) return;
    if (!PACKED && blockIdx.x + blockIdx.y == 0 && threadIdx.x == 0) p.meta[0] = p.meta[1] = 0;
    int64_t chain;
    int k;
    if (take_tile(p, chain, k)) scan_fwd_tile<x_t, l_t, h_t, V, PACKED>(p, chain, k, x, la, init, fin, h);
    if constexpr (PACKED) hand_on(p, init, fin);
}

template <typename x_t, typename l_t, typename h_t, int V, bool PACKED>
__device__ __forceinline__ void scan_bwd_tile(const Chain &p, int64_t chain, int k, const l_t *__restrict__ la,
                                              const h_t *__restrict__ h, const float *__restrict__ init,
                                              const h_t *__restrict__ dh, const float *__restrict__ dfin,
                                              x_t *__restrict__ dx, l_t *__restrict__ dla,
                                              float *__restrict__ dinit) {
    constexpr int LPR = kCw / V, G = kNt / LPR, TT = kElems / V;
    __shared__ float sA[G][kCw], sH[G][kCw];
    __shared__ int s_seq[PACKED ? kTc + 2 : 1];
    const int chunk = p.nchunk > 0 ? p.nchunk - 1 - k : 0;   // the chain runs from the last tile to the first
    const int row = (int)quotient(chain, p.ntile), col0 = (int)(chain - (int64_t)row * p.ntile) * kCw;
    const int tid = threadIdx.x, lp = tid % LPR, g = tid / LPR;
    const int t0 = chunk * kTc, len = min(kTc, p.T - t0);
    const bool live = col0 + lp * V < p.D;
    const int ch = min(col0 + lp * V, p.D - V);
    const int64_t base = ((int64_t)row * p.T + t0) * p.D;

    const int seq = PACKED ? load_seq(p, t0) : 0;
    Held<h_t, V> gr[TT], hr[TT];
    Gate<l_t, V> lr[TT];
    if (len > 0) {
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const int t = min(g * TT + i, len - 1);
            const uint32_t off = (uint32_t)t * (uint32_t)p.D + (uint32_t)ch;
            lr[i].load(la + base, off);
            gr[i].load(dh + base, off);
        }
        // h of the token before; at the very first token of a row it is not used
        const int back = t0 > 0 ? 0 : 1;
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const int t = max(min(g * TT + i, len - 1) - back, 0);
            hr[i].load(h + base - (1 - back) * (int64_t)p.D, (uint32_t)t * (uint32_t)p.D + (uint32_t)ch);
        }
    }
    const int wcol = col0 + tid / V * V;
    const int64_t wch = (int64_t)row * p.D + min(wcol, p.D - V) + tid % V;
    float edge = !PACKED && dfin && tid < kCw && wcol < p.D ? dfin[wch] : 0.f;
    uint32_t starts = 0, ends = 0;
    if constexpr (PACKED) {
        if (tid < kTc + 2) s_seq[tid] = seq;
        __syncthreads();
        edges<TT>(s_seq, g * TT, len, starts, ends);
    } else if (t0 == 0 && g == 0) {
        starts = 1;
    }
    if (len < kTc) {
#pragma unroll
        for (int i = 0; i < TT; ++i)
            if (g * TT + i >= len) {
                lr[i].zero();
                gr[i].zero();
            }
    }
    // behind a sequence's last token the gradient is its final state's
    auto enter = [&](int i, float (&e)[V]) {
        if constexpr (PACKED)
            if (ends >> i & 1) {
                const int64_t n = s_seq[g * TT + i + 1];
#pragma unroll
                for (int j = 0; j < V; ++j) e[j] = dfin && live ? dfin[n * p.D + ch + j] : 0.f;
            }
    };
    float A[V], H[V];
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = 1.f, H[j] = 0.f;
#pragma unroll
    for (int i = TT - 1; i >= 0; --i) {
        enter(i, H);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float a = lr[i].first(j);
            H[j] = a * (gr[i].get(j) + H[j]);
            A[j] *= a;
        }
    }
    mend_products(A, lr);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        sA[g][lp * V + j] = PACKED && ends ? kForgets : A[j];
        sH[g][lp * V + j] = H[j];
    }
    asm volatile("" : "+v"(edge));
    __syncthreads();
    if (tid < kCw) {
        float bA = 1.f, bH = 0.f;
#pragma unroll
        for (int q = G - 1; q >= 0; --q) join<PACKED>(bA, bH, sA[q][tid], sH[q][tid]);
        // a tile after this one, token by token
        auto map = [&](int tile, float &tA, float &tH) {
            const int from = (p.nchunk - 1 - tile) * kTc, to = min(from + kTc, p.T);
            const int c = (int)(wch - (int64_t)row * p.D);
            tA = 1.f, tH = 0.f;
#pragma nounroll
            for (int q = G - 1; q >= 0; --q) {
                float mA = 1.f, mH = 0.f;
                bool forget = false, nonzero = true;
#pragma nounroll
                for (int i = min(from + (q + 1) * TT, to) - 1; i >= from + q * TT; --i) {
                    const int64_t t = (int64_t)row * p.T + i;
                    if (PACKED && (i == p.T - 1 || p.seq[i + 1] != p.seq[i])) {
                        mH = dfin ? dfin[(int64_t)p.seq[i] * p.D + c] : 0.f;
                        forget = true;
                    }
                    const float a = exp_gate(to_f32(la[t * p.D + c]));
                    mH = a * (to_f32(dh[t * p.D + c]) + mH);
                    mA *= a;
                    nonzero &= a != 0.f;
                }
                join<PACKED>(tA, tH, PACKED && forget ? kForgets : above_zero(mA, nonzero), mH);
            }
        };
        float s = chain_state<PACKED>(p, chain, k, tid, bA, bH, edge, map);
#pragma unroll
        for (int q = G - 1; q >= 0; --q) {
            const float H = sH[q][tid];
            sH[q][tid] = s;
            s = apply<PACKED>(sA[q][tid], H, s);
        }
        if (!PACKED && dinit && wcol < p.D && chunk == 0) dinit[wch] = s;
    }
    __syncthreads();
    if (!live) return;
    float e[V];
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = sH[g][lp * V + j];
#pragma unroll
    for (int i = 0; i < TT; ++i) lr[i].touch(), gr[i].touch(), hr[i].touch();
#pragma unroll
    for (int i = TT - 1; i >= 0; --i) {
        const int t = g * TT + i;
        if (t >= len) continue;
        enter(i, e);
        const bool begin = starts >> i & 1;
        const int64_t n = PACKED ? s_seq[t + 1] : row;
        x_t ox[V];
        l_t ol[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float q = gr[i].get(j) + e[j];
            e[j] = lr[i].again(j) * q;
            float past = hr[i].get(j);
            if (begin) past = init ? init[n * p.D + ch + j] : 0.f;
            ox[j] = round_to<x_t>(q);
            ol[j] = round_to<l_t>(e[j] * past);
        }
        const uint32_t off = (uint32_t)t * (uint32_t)p.D + (uint32_t)ch;
        store_vec<x_t, V>(dx + base, off, ox);
        store_vec<l_t, V>(dla + base, off, ol);
        if constexpr (PACKED)
            if (dinit && begin)
#pragma unroll
                for (int j = 0; j < V; ++j) dinit[n * p.D + ch + j] = e[j];
    }
}

template <typename x_t, typename l_t, typename h_t, int V, bool PACKED>
__global__ __launch_bounds__(kNt, (min_waves<V, l_t, h_t, h_t>())) void scan_bwd_kernel(Chain p, const l_t *__restrict__ la,
                                                               const h_t *__restrict__ h,
                                                               const float *__restrict__ init,
                                                               const h_t *__restrict__ dh,
                                                               const float *__restrict__ dfin, x_t *__restrict__ dx,
                                                               l_t *__restrict__ dla, float *__restrict__ dinit) {
    if (PACKED && p.meta[1] != 0) return;
    if (!PACKED && blockIdx.x + blockIdx.y == 0 && threadIdx.x == 0) p.meta[0] = p.meta[1] = 0;
    int64_t chain;
    int k;
    if (take_tile(p, chain, k)) scan_bwd_tile<x_t, l_t, h_t, V, PACKED>(p, chain, k, la, h, init, dh, dfin, dx, dla, dinit);
    if constexpr (PACKED) hand_on(p, dfin, dinit);
}

// ---- short rows --------------------------------------------------------------------
//
// Batches of many short rows: one thread takes V channels of a row from its
// first token to its last, kBatch tokens in flight at a time.  No joins and no
// hand-overs, and no lane waits for a tile that the row does not fill.
constexpr int kBatch = 8;

template <typename x_t, typename l_t, typename h_t, int V>
__global__ __launch_bounds__(256) void scan_fwd_rows_kernel(int64_t rows, int T, int D, int32_t *__restrict__ meta,
                                                            const x_t *__restrict__ x, const l_t *__restrict__ la,
                                                            const float *init, float *fin, h_t *__restrict__ h) {
    if (blockIdx.x == 0 && threadIdx.x == 0) meta[0] = meta[1] = 0;
    const int per = (D + V - 1) / V;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * per; i += (int64_t)gridDim.x * 256) {
        const int64_t row = quotient(i, per);
        const int ch = min((int)(i - row * per) * V, D - V);   // the last thread ends with the row, as in a tile
        const int64_t base = row * T * D + ch, at = row * D + ch;
        float s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = init ? init[at + j] : 0.f;
        for (int t0 = 0; t0 < T; t0 += kBatch) {
            Held<x_t, V> xr[kBatch];
            Held<l_t, V> lr[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const uint32_t off = (uint32_t)min(t0 + q, T - 1) * (uint32_t)D;
                lr[q].load(la + base, off);
                xr[q].load(x + base, off);
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (t0 + q >= T) break;
                h_t o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    s[j] = fmaf(exp_gate(lr[q].get(j)), s[j], xr[q].get(j));
                    o[j] = round_to<h_t>(s[j]);
                }
                store_vec<h_t, V>(h + base, (uint32_t)(t0 + q) * (uint32_t)D, o);
            }
        }
        if (fin)
#pragma unroll
            for (int j = 0; j < V; ++j) fin[at + j] = s[j];
    }
}

template <typename x_t, typename l_t, typename h_t, int V>
__global__ __launch_bounds__(256) void scan_bwd_rows_kernel(int64_t rows, int T, int D, int32_t *__restrict__ meta,
                                                            const l_t *__restrict__ la, const h_t *__restrict__ h,
                                                            const float *__restrict__ init,
                                                            const h_t *__restrict__ dh,
                                                            const float *__restrict__ dfin, x_t *__restrict__ dx,
                                                            l_t *__restrict__ dla, float *__restrict__ dinit) {
    if (blockIdx.x == 0 && threadIdx.x == 0) meta[0] = meta[1] = 0;
    const int per = (D + V - 1) / V;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * per; i += (int64_t)gridDim.x * 256) {
        const int64_t row = quotient(i, per);
        const int ch = min((int)(i - row * per) * V, D - V);
        const int64_t base = row * T * D + ch, at = row * D + ch;
        float e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = dfin ? dfin[at + j] : 0.f;
        for (int t0 = T - 1; t0 >= 0; t0 -= kBatch) {
            Held<l_t, V> lr[kBatch];
            Held<h_t, V> gr[kBatch], hr[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int t = max(t0 - q, 0);
                lr[q].load(la + base, (uint32_t)t * (uint32_t)D);
                gr[q].load(dh + base, (uint32_t)t * (uint32_t)D);
                hr[q].load(h + base, (uint32_t)max(t - 1, 0) * (uint32_t)D);
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int t = t0 - q;
                if (t < 0) break;
                x_t ox[V];
                l_t ol[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float g = gr[q].get(j) + e[j];
                    e[j] = exp_gate(lr[q].get(j)) * g;
                    const float past = t > 0 ? hr[q].get(j) : init ? init[at + j] : 0.f;
                    ox[j] = round_to<x_t>(g);
                    ol[j] = round_to<l_t>(e[j] * past);
                }
                store_vec<x_t, V>(dx + base, (uint32_t)t * (uint32_t)D, ox);
                store_vec<l_t, V>(dla + base, (uint32_t)t * (uint32_t)D, ol);
            }
        }
        if (dinit)
#pragma unroll
            for (int j = 0; j < V; ++j) dinit[at + j] = e[j];
    }
}

// Rows of at most 32 tokens with a thread for every lane of the GPU, or of one
// batch.  Measured in bf16 at D = 1024, rows and tiles, in us:
//                 forward      gradient
//   4096 x  8     39   199     57   322
//   1024 x 16     19    54     30    90
//    512 x 32     26    31     32    52
//    256 x 32     23    18     21    27
//    256 x 16     12    16     13    24
//    128 x 32     19    11     15    15
//    512 x 64     51    40     65    71
// and 11 and 11, 13 and 13 at 4 x 8, which is the call's own time.  At the border of
// the rule, 256 x 32, the forward pass loses 5 us and the gradient gains 7: one
// rule stands for both.
static bool short_rows(const ScanArgs &a) {
    return !a.cu_seqlens && a.T > 0 &&
           (a.T <= kBatch || (a.T <= kShortRow && (int64_t)a.B * a.D >= 256 * 1024));
}

static int scan_patience() {
    const char *s = getenv("GDN_SCAN_PATIENCE");
    return s && *s ? std::max(atoi(s), 0) : kPatience;
}

// Fills `c` and enqueues the setup kernel where the call needs one.
// `init`: the initial states that the kernel reads.
static hipError_t scan_setup(const ScanArgs &a, Chain &c, const float *&init, hipStream_t st) {
    const bool packed = a.cu_seqlens != nullptr;
    const auto w = scan_workspace_layout(a.B, a.T, a.D, a.N, packed);
    char *ws = static_cast<char *>(a.workspace);
    c.T = a.T, c.D = a.D, c.N = a.N, c.nchunk = (int)w.chunks, c.ntile = (int)w.tiles;
    c.cu = a.cu_seqlens;
    c.meta = reinterpret_cast<int32_t *>(ws);
    c.seq = reinterpret_cast<int32_t *>(ws + w.off_seq);
    c.patience = scan_patience();
    c.agg = reinterpret_cast<uint64_t *>(ws + w.off_agg);
    c.grp = reinterpret_cast<uint64_t *>(ws + w.off_grp);
    c.pre = reinterpret_cast<uint64_t *>(ws + w.off_pre);
    c.nchain = w.rows * w.tiles;
    c.blocks = (w.chunks > 0 ? w.chunks : 1) * c.nchain;
    init = a.init_state;
    float *keep = reinterpret_cast<float *>(ws + w.off_init);
    const bool over = keeps_init(packed, a.D, w.chunks) && init && init == a.final_state;
    if (over) init = keep;
    if (w.chunks <= 1 && !packed && !over) return hipSuccess;
    const int64_t words16 = (int64_t)(w.total - w.off_agg) / 16;
    const int64_t other = std::max<int64_t>(over ? (int64_t)a.N * a.D : 0, packed ? a.T : 0);
    const int64_t work = std::max(words16, other);
    int64_t blocks = (work + 255) / 256;
    blocks = blocks < 1 ? 1 : (blocks > 2048 ? 2048 : blocks);
    ProfScope prof("gdn_scan_setup", st);
    scan_setup_kernel<<<(unsigned)blocks, 256, 0, st>>>(a.N, a.T, a.cu_seqlens, c.meta,
                                                        reinterpret_cast<int32_t *>(ws + w.off_seq),
                                                        reinterpret_cast<u32x4_t *>(ws + w.off_agg), words16,
                                                        a.init_state, keep, over ? (int64_t)a.N * a.D : 0);
    return hipGetLastError();
}

// Loads of 4 channels, of one where there are fewer.  Rows start on any
// element: the vectors need no alignment beyond the element's.  One channel at
// a time takes the gradient past its registers (3 to 38 of a thread's are in
// scratch; 64 x 4096 x 3 in fp32 39 us); at four, fp32 h leaves 2 to 16 there,
// which costs nothing that shows (337 us above).
template <typename F>
static hipError_t with_shape(const ScanArgs &a, F f) {
    using std::integral_constant;
    const bool packed = a.cu_seqlens != nullptr;
    auto vec = [&](auto v) {
        return packed ? f(v, integral_constant<bool, true>{}) : f(v, integral_constant<bool, false>{});
    };
    return a.D >= 4 ? vec(integral_constant<int, 4>{}) : vec(integral_constant<int, 1>{});
}

// A block for each tile, and packed for each sequence up to 2048: empty sequences
// are shared out over the blocks (hand_on).  4096 sequences, 16 of them with a
// token, x 128 channels, one tile: 1015 us with its one block, 19 us so.
static dim3 scan_grid(const ScanArgs &a, const Chain &c) {
    const int64_t n = a.cu_seqlens ? std::max<int64_t>(c.blocks, std::min(a.N, 2048)) : c.blocks;
    return dim3((unsigned)std::min(n, kMaxGridX), (unsigned)scan_tiles(n, kMaxGridX));
}

hipError_t launch_scan_fwd(const ScanArgs &a, hipStream_t st) {
    Chain c;
    const float *init;
    hipError_t e = scan_setup(a, c, init, st);
    if (e != hipSuccess) return e;
    const dim3 blocks = scan_grid(a, c);
    ProfScope prof("gdn_scan_fwd", st);
    return with_types(a.in_dtype, a.gate_dtype, a.out_dtype, [&](auto x, auto l, auto h) {
        return with_shape(a, [&](auto v, auto packed) {
            using x_t = decltype(x);
            using l_t = decltype(l);
            using h_t = decltype(h);
            constexpr int V = decltype(v)::value;
            if constexpr (!decltype(packed)::value) {
                if (short_rows(a)) {
                    const int64_t threads = a.B * scan_tiles(a.D, V);
                    scan_fwd_rows_kernel<x_t, l_t, h_t, V>
                        <<<(unsigned)std::min<int64_t>(scan_tiles(threads, 256), 1 << 20), 256, 0, st>>>(
                    a.B, a.T, a.D, c.meta, static_cast<const x_t *>(a.x), static_cast<const l_t *>(a.log_alpha), init, a.final_state, static_cast<h_t *>(a.h));
                    return hipGetLastError();
                }
            }
            scan_fwd_kernel<x_t, l_t, h_t, V, decltype(packed)::value>
                <<<blocks, kNt, 0, st>>>(c, static_cast<const x_t *>(a.x),
                                                   static_cast<const l_t *>(a.log_alpha), init, a.final_state,
                                                   static_cast<h_t *>(a.h));
            return hipGetLastError();
        });
    });
}

hipError_t launch_scan_bwd(const ScanArgs &a, hipStream_t st) {
    Chain c;
    const float *init;
    hipError_t e = scan_setup(a, c, init, st);
    if (e != hipSuccess) return e;
    const dim3 blocks = scan_grid(a, c);
    ProfScope prof("gdn_scan_bwd", st);
    return with_types(a.in_dtype, a.gate_dtype, a.out_dtype, [&](auto x, auto l, auto h) {
        return with_shape(a, [&](auto v, auto packed) {
            using x_t = decltype(x);
            using l_t = decltype(l);
            using h_t = decltype(h);
            constexpr int V = decltype(v)::value;
            if constexpr (!decltype(packed)::value) {
                if (short_rows(a)) {
                    const int64_t threads = a.B * scan_tiles(a.D, V);
                    scan_bwd_rows_kernel<x_t, l_t, h_t, V>
                        <<<(unsigned)std::min<int64_t>(scan_tiles(threads, 256), 1 << 20), 256, 0, st>>>(
                    a.B, a.T, a.D, c.meta, static_cast<const l_t *>(a.log_alpha), static_cast<const h_t *>(a.h), init, static_cast<const h_t *>(a.d_h),
                    a.d_final, static_cast<x_t *>(a.dx), static_cast<l_t *>(a.dlog_alpha), a.d_init);
                    return hipGetLastError();
                }
            }
            scan_bwd_kernel<x_t, l_t, h_t, V, decltype(packed)::value>
                <<<blocks, kNt, 0, st>>>(c, static_cast<const l_t *>(a.log_alpha),
                                                   static_cast<const h_t *>(a.h), init,
                                                   static_cast<const h_t *>(a.d_h), a.d_final,
                                                   static_cast<x_t *>(a.dx), static_cast<l_t *>(a.dlog_alpha),
                                                   a.d_init);
            return hipGetLastError();
        });
    });
}

// ---- single step -----------------------------------------------------------------

// Four elements a thread (the arrays are dense and 16-byte aligned).  At 256 x
// 2048 the call is bound by its launch.
template <typename x_t, typename l_t, typename h_t>
__global__ __launch_bounds__(256) void scan_step_kernel(int64_t n, float *__restrict__ state,
                                                        const x_t *__restrict__ x, const l_t *__restrict__ la,
                                                        h_t *__restrict__ h) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
        if (i + 4 <= n) {
            Held<x_t, 4> xr;
            Held<l_t, 4> lr;
            lr.load(la + i, 0);
            xr.load(x + i, 0);
            float4_t s = *reinterpret_cast<const float4_t *>(state + i);
            h_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = fmaf(exp_gate(lr.get(j)), s[j], xr.get(j));
                o[j] = round_to<h_t>(s[j]);
            }
            *reinterpret_cast<float4_t *>(state + i) = s;
            store_vec<h_t, 4>(h + i, 0, o);
        } else {
            for (int64_t e = i; e < n; ++e) {
                const float s = fmaf(exp_gate(to_f32(la[e])), state[e], to_f32(x[e]));
                state[e] = s;
                h[e] = round_to<h_t>(s);
            }
        }
    }
}

hipError_t launch_scan_step(const ScanStepArgs &a, hipStream_t st) {
    const int64_t n = (int64_t)a.N * a.D;
    const unsigned blocks = (unsigned)std::min<int64_t>(scan_tiles(n, 1024), 1 << 20);
    ProfScope prof("gdn_scan_step", st);
    return with_types(a.in_dtype, a.gate_dtype, a.out_dtype, [&](auto x, auto l, auto h) {
        using x_t = decltype(x);
        using l_t = decltype(l);
        using h_t = decltype(h);
        scan_step_kernel<x_t, l_t, h_t><<<blocks, 256, 0, st>>>(n, a.state, static_cast<const x_t *>(a.x),
                                                                static_cast<const l_t *>(a.log_alpha),
                                                                static_cast<h_t *>(a.h));
        return hipGetLastError();
    });
}

}  // namespace gdn
