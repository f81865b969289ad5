// Windowed attention with sinks, backward.  With P = exp(s - lse) over the visible
// pairs and D_i = d_o_i o_i,
//   dV = P^T dO      dP = dO V^T      dS = P (dP - D)
//   dQ = scale dS K  dK = scale dS^T Q
// Two kernels, so that every sum has one owner and a fixed order, without atomics;
// S and dP are formed in both (7 products of the visible pairs' size instead of 5).
//
// Query side: a wave owns 32 rows (query token, head of the group) and walks over
// the keys that they see, as forward: S^T and dP^T as 32 x 32 tiles with a row in
// each lane, dS^T as it lies the operand of dQ^T += K^T dS^T.
//
// Key side: a wave owns 32 keys and walks over the rows that see them: S and dP
// with a key in each lane, P and dS the operands of dV^T += dO^T P and
// dK^T += Q^T dS.  All later tokens see the sinks: what lies past the window of the
// first key tile is cut into parts, each a block of its own whose share of the sinks'
// gradients goes to the workspace in fp32, and a last kernel adds the parts.
//
// Measured (MI355X): 4 x 4096 tokens, 16 heads on 4 of 128, window 2048, 4 sinks, bf16: query
// side 295 to 300 us (1.05 PFLOP/s over its three products, the matrix cores busy 52%), key side
// 610 to 630 (0.82 over its five, busy 35%).  32768 tokens, 16 heads on 8 of 64, 16 sinks,
// fp16: 456 to 468 and 695 to 740.  The first case in fp32: 3.0 and 5.8 ms with one wave a
// SIMD, 3.4 and 6.75 with two, which spill; with 64-wide heads 1.27 and 2.19.  Both are bound
// by what two waves a SIMD overlap of products, exponentials and LDS reads; the key side
// also has two or three times as many units of unequal length as blocks fit.  Key side, of the same first case: far parts of the
// sinks without masks 965 -> 757 us, no looks for values that are not finite in masked
// tiles 757 -> 614, reads in batches 650 -> 628 (another GPU).
#include "gdn_ops.h"
#include "gdn_swa.h"

#include <algorithm>

namespace gdn {

constexpr int kKeys = 64;            // keys of a staged tile, query side
constexpr int kRows = 64;            // rows of a staged tile, key side

// In one rounding, so that all places that take it have the same bits.
__device__ __forceinline__ float log2_lse(float lse, float lift = 0.f) {
    // a row that saw nothing: every probability 0
    return lse == -__builtin_inff() ? __builtin_inff() : fmaf(lse, 1.4426950408889634f, -lift);
}

// fp16 holds dS only from 2^-24 to 65504, and many small ones may make up dQ and dK (of
// 32768 keys and 2^-10 of d_o, dQ was 3.7% off).  It is taken times a power of two per row of
// dQ or dK, at first 2^64, lowered with the sums so far where an element comes near the
// end of fp16's range; the store takes it out again.  Lowered to [2^12, 2^13), so that
// the next larger ones seldom ask for it again: elements down to 2^-26 of the largest are
// rounded once.  Measured, 32768 tokens, 16 heads on 8 of 64, query and key side:
// 447 and 699 us with dS as it is, 468 and 720 so; 4 x 4096 tokens, 16 heads on 4 of 128, 320
// and 652, 335 and 681.
constexpr int kLiftDs = 64;
constexpr float kMostDs = 60000.f;
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// By how many powers an element of size t has to be lowered.
__device__ __forceinline__ int lower_ds(float t) { return t < kMostDs ? 0 : (int)(__float_as_uint(t) >> 23) - 139; }
__device__ __forceinline__ float inverse_power(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

template <typename T, int D, int NW>
__global__ __launch_bounds__(64 * NW, (Rows<T, D>::RB >= 512 ? 1 : 2)) void swa_dq_kernel(
    SwaShape sh, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, const T *__restrict__ o,
    const float *__restrict__ lse, const T *__restrict__ d_o, T *__restrict__ dq, float *__restrict__ dsum) {
    using R = Rows<T, D>;
    constexpr int RB = R::RB, TILE = kKeys * RB, PIECES = TILE / 1024 / NW;
    extern __shared__ __align__(16) char smem[];   // two stages of K and V tiles
    SwaUnit u;
    if (!swa_find(sh, true, u)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, h = l >> 5;
    const int shift = u.Lk - u.Lq;
    const int t0 = u.unit * sh.tokens, t1 = min(t0 + sh.tokens, u.Lq);
    const int pfirst = t0 + shift, plast = t1 - 1 + shift;
    const int W = sh.window;

    const int row = wave * 32 + (l & 31), tt = row / sh.G, token = t0 + tt;
    const bool on = tt < sh.tokens && token < t1;
    const int pos = min(token, t1 - 1) + shift;
    const int w0 = t0 + wave * 32 / sh.G;
    const bool busy = w0 < t1 && wave * 32 / sh.G < sh.tokens;
    const int p0 = w0 + shift, p1 = min(t0 + (wave * 32 + 31) / sh.G, t1 - 1) + shift;
    const int64_t at = (u.q0 + min(token, t1 - 1)) * sh.H + u.hk * sh.G + row % sh.G;
    u32x4_t qf[R::NS], gf[R::NS];
    float dd = 0.f;
#pragma unroll
    for (int s = 0; s < R::NS; ++s) {
        const int64_t b = at * RB + 32 * s + 16 * h;
        qf[s] = *reinterpret_cast<const u32x4_t *>(reinterpret_cast<const char *>(q) + b);
        gf[s] = *reinterpret_cast<const u32x4_t *>(reinterpret_cast<const char *>(d_o) + b);
        const u32x4_t of = *reinterpret_cast<const u32x4_t *>(reinterpret_cast<const char *>(o) + b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (R::F32) {
                dd = fmaf(__uint_as_float(of[e]), __uint_as_float(gf[s][e]), dd);
            } else {
                dd = fmaf(R::half_of(of[e]), R::half_of(gf[s][e]), dd);
                dd = fmaf(R::half_of(of[e] >> 16), R::half_of(gf[s][e] >> 16), dd);
            }
        }
    }
    dd = half_sum(dd);
    if (on && h == 0) dsum[at] = dd;
    float lse2 = log2_lse(lse[at]);
    arrived(lse2);
    constexpr bool LIFT = std::is_same_v<T, _Float16>;
    float unit, base;                              // of dS; lse2 less its log2
#pragma unroll
    for (int s = 0; s < R::NS; ++s) arrived(qf[s]), arrived(gf[s]);

    int low = max(pfirst - W + 1, 0);
    const int high = plast + 1;
    if (low <= sh.sinks) low = 0;
    const int ns = low > 0 ? (sh.sinks + kKeys - 1) / kKeys : 0;
    const int tiles = high > low ? ns + (high - low + kKeys - 1) / kKeys : 0;
    // Tiles that every row of the block sees whole come first, then those that the mask
    // cuts: a loop each, so that either keeps its registers.
    const int whole_a = ns + max(plast - W + kKeys - low, 0) / kKeys;   // the first that no row's window begins in
    const int whole = max(ns + (pfirst + 1 - low) / kKeys - whole_a, 0);
    auto tile_at = [&](int x) { return x < whole ? whole_a + x : x - whole < whole_a ? x - whole : x; };
    auto first_key = [&](int it) { return it < ns ? it * kKeys : low + (it - ns) * kKeys; };

    const uint32_t stride = (uint32_t)sh.KV * RB;
    const int64_t head = (u.k0 * sh.KV + u.hk) * (int64_t)RB;
    uint32_t off[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int b = (i * NW + wave) * 1024 + l * 16;
        off[i] = b / RB * stride + R::chunk_at(b) * 16;
    }
    const uint32_t lds = lds_addr(smem) + wave * 1024;
    auto load = [&](int it) {
        const int j0 = first_key(tile_at(it)), n = min(u.Lk - j0, kKeys);
        const int64_t b = head + (int64_t)j0 * stride;
        const uint32_t bytes = (n - 1) * stride + RB;
        const uint32_t to = lds + (it & 1) * 2 * TILE;
        stage<PIECES, NW * 1024>(reinterpret_cast<const char *>(k) + b, bytes, off, to);
        stage<PIECES, NW * 1024>(reinterpret_cast<const char *>(v) + b, bytes, off, to + TILE);
    };

    f32x16_t acc[R::ND];
    const typename R::Lane lane;
    // All tiles, and as forward a second time where the sums are not finite.
    auto walk = [&](auto careful) {
        constexpr bool CAREFUL = decltype(careful)::value;
#pragma unroll
        for (int dt = 0; dt < R::ND; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[dt][i] = 0.f;
        unit = LIFT ? power_of_2(kLiftDs) : 1.f, base = LIFT ? lse2 - kLiftDs : lse2;
        // One staged tile after the other, [x0, x1) of their order.
        auto each = [&](int x0, int x1, auto body) {
            for (int x = x0; x < x1; ++x) {
                staged_barrier();
                if (x + 1 < tiles) load(x + 1);
                if (busy) body(tile_at(x), smem + (x & 1) * 2 * TILE);
            }
        };
        auto process = [&](auto masked, const char *kt, int j0, int jend, int r0) {
            const char *vt = kt + TILE;
            constexpr bool MASK = decltype(masked)::value;
            const typename R::Lane ln = lane.fresh();
            f32x16_t S, P;
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i] = P[i] = 0.f;
#pragma unroll
            for (int s = 0; s < R::NS; ++s) {
                mma32<T>(S, R::frag(kt, ln, r0, s), qf[s]);
                mma32<T>(P, R::frag(vt, ln, r0, s), gf[s]);
            }
            uint32_t seen = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = __builtin_amdgcn_exp2f(fmaf(S[i], sh.c, -base)) * (P[i] - dd);
                if constexpr (MASK) {
                    const int j = j0 + r0 + 4 * (ln.l >> 5) + 8 * (i >> 2) + (i & 3);
                    bool see = j <= pos && j < jend && (j > pos - W || j < sh.sinks);
                    if constexpr (CAREFUL) see &= lse2 != __builtin_inff();   // a row without weights has no gradient
                    S[i] = see ? x : 0.f;
                    seen |= (uint32_t)see << i;
                } else {
                    S[i] = x;
                }
            }
            if constexpr (LIFT) {
                float t = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) t = fmaxf(t, fabsf(S[i]));
                if (__any(t >= kMostDs)) {
                    const int less = lower_ds(half_max(t));
                    const float f = power_of_2(-less);
                    unit *= f;
                    base += less;
                    S *= f;
#pragma unroll
                    for (int dt = 0; dt < R::ND; ++dt) acc[dt] *= f;
                }
            }
            if constexpr (CAREFUL) R::add_seen(acc, kt, ln, r0, S, seen);
            else R::add(acc, kt, ln, r0, S);
        };
        if (tiles) load(0);
        if constexpr (!CAREFUL)
            each(0, whole, [&](int it, const char *kt) {
#pragma unroll
                for (int r0 = 0; r0 < kKeys; r0 += 32) process(std::false_type{}, kt, first_key(it), 0, r0);
            });
        each(CAREFUL ? 0 : whole, tiles, [&](int it, const char *kt) {
            const int j0 = first_key(it), jend = it < ns ? sh.sinks : high;
#pragma unroll 1
            for (int r0 = 0; r0 < kKeys; r0 += 32) {
                const int j = j0 + r0;           // 32 keys that no row of the wave sees are left out
                if (j > p1 || j >= jend || (j + 31 <= p0 - W && j >= sh.sinks)) continue;
                process(std::true_type{}, kt, j0, jend, r0);
            }
        });
    };
    walk(std::false_type{});
    if (__syncthreads_or(busy && any_not_finite(acc))) walk(std::true_type{});
    if (busy) store_column<T, D>(dq + at * D, acc, LIFT ? sh.scale * inverse_power(unit) : sh.scale, on);
}

// Where the far parts of a sequence begin: tokens from `reach` on are past the
// window of the first key tile.
struct FarParts {
    int reach, parts;
};
__host__ __device__ __forceinline__ FarParts far_parts(int Lq, int Lk, int window, int sinks, int far) {
    const int64_t reach = (int64_t)kSwaKeyTile + window - 1 - (Lk - (int64_t)Lq);
    FarParts f;
    f.reach = (int)(reach < 0 ? 0 : reach > Lq ? Lq : reach);
    f.parts = sinks && Lk > 0 ? (Lq - f.reach + far - 1) / far : 0;
    return f;
}
// First part in the workspace of a sequence that has any: part 0 is the near one's.  Its keys are
// then `far` or more, and its parts at most keys / far: with the near one not more than
// twice that, so by its first key no two sequences share a place.
__device__ __forceinline__ int64_t far_first(int64_t k0, int far) { return 2 * (k0 / far); }

// The two accumulators and the operands K and V of a wave are 3 D 32-bit registers
// in 16 bits, 4 D in fp32.  Where that leaves too few of 256, dV and dK are made by
// different blocks, the second with S once more (5 products instead of 4).
// Measured, 4 x 4096 tokens, 16 heads on 4 of 128, window 2048, in bf16: different blocks
// 1118 us, one block for both 3715 with two waves a SIMD (registers spill) and 1195 with
// one; since then the split form has come to 610 to 630.  4096 tokens, 16 heads on 8 of 64,
// in fp32: 817 us split, 684 not.
template <typename T, int D>
constexpr bool kSplitKeySide = D == 128;

template <typename T, int D>
__global__ __launch_bounds__(256, (Rows<T, D>::RB >= 512 ? 1 : 2)) void swa_dkv_kernel(
    SwaShape sh, int far, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
    const float *__restrict__ lse, const T *__restrict__ d_o, const float *__restrict__ dsum, T *__restrict__ dk,
    T *__restrict__ dv, float *__restrict__ share) {
    using R = Rows<T, D>;
    constexpr int NW = 4, RB = R::RB, TILE = kRows * RB, PIECES = TILE / 1024 / NW;
    extern __shared__ __align__(16) char smem[];   // two stages of Q and dO tiles, of lse and D
    float *stats = reinterpret_cast<float *>(smem + 4 * TILE);
    int *tokens = reinterpret_cast<int *>(stats + 4 * kRows);   // of a tile's rows, from its first on
    SwaUnit u;
    if (!swa_find<kSplitKeySide<T, D> ? 2 : 1>(sh, false, u)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, h = l >> 5;
    const int shift = u.Lk - u.Lq, W = sh.window;
    const FarParts fp = far_parts(u.Lq, u.Lk, W, sh.sinks, far);
    const int part = u.unit < fp.parts ? u.unit : -1;   // >= 0: a far part; these come first
    const int jt = part >= 0 ? 0 : (u.unit - fp.parts) * kSwaKeyTile;

    // the tokens that this block takes
    int ta, tb;
    if (part >= 0) {
        ta = fp.reach + part * far;
        tb = min(ta + far, u.Lq);
    } else {
        ta = max(jt - shift, 0);
        tb = (int)min((int64_t)jt + kSwaKeyTile - 1 + W - shift, (int64_t)u.Lq);
    }
    const int tiles = tb > ta ? (tb - ta + sh.tokens - 1) / sh.tokens : 0;

    const int k0 = jt + wave * 32, key = k0 + (l & 31);
    const bool busy = k0 < u.Lk && (part < 0 || k0 < sh.sinks);
    const int64_t at = (u.k0 + min(key, u.Lk - 1)) * sh.KV + u.hk;
    u32x4_t kf[R::NS], vf[R::NS];
#pragma unroll
    for (int s = 0; s < R::NS; ++s) {
        const int64_t b = at * RB + 32 * s + 16 * h;
        kf[s] = *reinterpret_cast<const u32x4_t *>(reinterpret_cast<const char *>(k) + b);
        vf[s] = *reinterpret_cast<const u32x4_t *>(reinterpret_cast<const char *>(v) + b);
    }
#pragma unroll
    for (int s = 0; s < R::NS; ++s) arrived(kf[s]), arrived(vf[s]);

    // rows left over of a tile (the group's size does not divide it) are never
    // copied: they stay zeros, and their probabilities 0
    const int rows = sh.tokens * sh.G;
    const int half = 32 / sh.G, half_end = min(31 / sh.G + 1, sh.tokens);   // tokens of rows 32 .. and to row 31
    if (threadIdx.x < kRows) tokens[threadIdx.x] = (int)threadIdx.x < rows ? (int)threadIdx.x / sh.G : 1 << 30;
    if (rows < kRows) {
        for (int b = threadIdx.x * 16; b < (kRows - rows) * RB; b += 256 * 16)
#pragma unroll
            for (int x = 0; x < 4; ++x) *reinterpret_cast<u32x4_t *>(smem + x * TILE + rows * RB + b) = u32x4_t{0u, 0u, 0u, 0u};
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    const uint32_t stride = (uint32_t)sh.H * RB;
    uint32_t off[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int b = (i * NW + wave) * 1024 + l * 16, r = b / RB;
        off[i] = r < rows ? (r / sh.G) * stride + (r % sh.G) * RB + R::chunk_at(b) * 16 : 0xFFFFFFFFu;
    }
    const uint32_t lds = lds_addr(smem) + wave * 1024;
    // Tiles whose rows all see all keys of the block come first, then those that the mask
    // cuts.  Neighbouring key tiles see almost the same tokens, 128 later each: they take
    // the first kind in the order of the tokens' residues, so that blocks that run
    // side by side read the same rows at about the same time, out of one L2.
    // Of a far part every full tile is of the first kind: its rows see the sinks, and
    // the gradients of other keys are dropped.
    int whole_a = 0, whole = (tb - ta) / sh.tokens;
    if (part < 0) {
        whole_a = max(jt + kSwaKeyTile - 1 - shift - ta + sh.tokens - 1, 0) / sh.tokens;
        const int64_t end = min((int64_t)jt + W - shift, (int64_t)tb) - ta;
        whole = max((int)max(end, (int64_t)0) / sh.tokens - whole_a, 0);
    }
    const int turn = whole ? (whole - (ta / sh.tokens + whole_a) % whole) % whole : 0;
    auto first_token = [&](int x) {
        const int y = x + turn < whole ? x + turn : x + turn - whole;
        return ta + (x < whole ? whole_a + y : x - whole < whole_a ? x - whole : x) * sh.tokens;
    };
    const int srow = l, stoken = srow / sh.G;      // waves 0 and 1 bring lse and D of the tile's rows
    float stat = 0.f;
    // dV takes fp16 probabilities times 2^15: the small ones, which many rows may share, would
    // be subnormal or 0
    constexpr bool LIFT = std::is_same_v<T, _Float16>;
    const int lift = LIFT && (!kSplitKeySide<T, D> || u.role == 0) ? 15 : 0;
    constexpr float UNLIFT = LIFT ? 0x1p-15f : 1.f;
    auto load = [&](int it) {
        const int t0 = first_token(it), n = min(tb - t0, sh.tokens);
        const int64_t first = (u.q0 + t0) * sh.H + u.hk * sh.G, b = first * RB;
        const uint32_t bytes = (n - 1) * stride + sh.G * RB;
        const uint32_t to = lds + (it & 1) * 2 * TILE;
        stage<PIECES, NW * 1024>(reinterpret_cast<const char *>(q) + b, bytes, off, to);
        stage<PIECES, NW * 1024>(reinterpret_cast<const char *>(d_o) + b, bytes, off, to + TILE);
        if (wave < 2) {
            const bool there = srow < rows && stoken < n;
            const int64_t a = first + (there ? (int64_t)stoken * sh.H + srow % sh.G : 0);
            stat = wave == 0 ? log2_lse(lse[a], lift) : LIFT ? -dsum[a] : dsum[a];
            if (!there) stat = wave == 0 ? __builtin_inff() : 0.f;
        }
    };
    auto put = [&](int it) {
        if (wave < 2) stats[((it & 1) * 2 + wave) * kRows + l] = stat;
    };

    const typename R::Lane lane;
    float unit = 1.f;                              // of dS
    // All tiles of rows, for dV, dK or both.
    auto walk = [&](auto careful, auto make_v, auto make_k, f32x16_t (&av)[R::ND], f32x16_t (&ak)[R::ND]) {
        constexpr bool CAREFUL = decltype(careful)::value, MAKE_V = decltype(make_v)::value,
                       MAKE_K = decltype(make_k)::value;
#pragma unroll
        for (int dt = 0; dt < R::ND; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (MAKE_K) ak[dt][i] = 0.f;
                if (MAKE_V) av[dt][i] = 0.f;
            }
        // what other lanes of a far part make is dropped
        if constexpr (LIFT) unit = part < 0 || key < sh.sinks ? power_of_2(kLiftDs) : 0.f;
        // The unit follows a tile's largest dS; returns by what its elements are to be lowered.
        auto lower = [&](float t) {
            const float f = power_of_2(-lower_ds(half_max(t)));
            unit *= f;
#pragma unroll
            for (int dt = 0; dt < R::ND; ++dt) ak[dt] *= f;
            return f;
        };
        // CAREFUL: `look` asks for the largest dS of each key alone, and the unit follows it
        // before the sums are made.
        float peak = 0.f;
        auto process = [&](auto subs, auto masked, auto looks, int x, int t0, int r0) {
            const char *qt = smem + (x & 1) * 2 * TILE, *gt = qt + TILE;
            const float *st = stats + (x & 1) * 2 * kRows;
            constexpr int NSUB = decltype(subs)::value;
            constexpr bool MASK = decltype(masked)::value, LOOK = decltype(looks)::value;
            const typename R::Lane ln = lane.fresh();
            const float *sr = st + r0 + 4 * (ln.l >> 5);
            f32x16_t S[NSUB], P[NSUB];
#pragma unroll
            for (int n = 0; n < NSUB; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) S[n][i] = P[n][i] = 0.f;
            R::dot(S, qt, ln, r0, kf);
            uint32_t seen = 0;
#pragma unroll
            for (int a = 0; a < 4 * NSUB; ++a) {
                const float4_t L = *reinterpret_cast<const float4_t *>(sr + 8 * a);
                int4 to{};
                if constexpr (MASK) to = *reinterpret_cast<const int4 *>(tokens + (sr - st) + 8 * a);
                const int tok[4] = {to.x, to.y, to.z, to.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 4 * (a & 3) + e;
                    float p = S[a >> 2][i];
                    p = __builtin_amdgcn_exp2f(fmaf(p, sh.c, -L[e]));
                    if constexpr (MASK) {
                        const int token = t0 + tok[e], pos = token + shift;
                        bool see = token < tb && key <= pos && (key > pos - W || key < sh.sinks);
                        if constexpr (CAREFUL) see &= L[e] != __builtin_inff();
                        p = see ? p : 0.f;
                        seen |= (uint32_t)see << i;
                    }
                    S[a >> 2][i] = p;
                }
            }
            if constexpr (MAKE_V && !LOOK) {
                if constexpr (CAREFUL) {
                    R::add_seen(av, gt, ln, r0, S[0], seen);
                } else {
#pragma unroll
                    for (int n = 0; n < NSUB; ++n) R::add(av, gt, ln, r0 + 32 * n, S[n]);
                }
            }
            if constexpr (!MAKE_K) return;
            if constexpr (LIFT) {                  // dP - D at once, for the product that the power of two costs
#pragma unroll
                for (int a = 0; a < 4 * NSUB; ++a) {
                    const float4_t dd = *reinterpret_cast<const float4_t *>(sr + kRows + 8 * a);
#pragma unroll
                    for (int e = 0; e < 4; ++e) P[a >> 2][4 * (a & 3) + e] = dd[e];
                }
            }
            R::dot(P, gt, ln, r0, vf);
#pragma unroll
            for (int a = 0; a < 4 * NSUB; ++a) {
                float4_t dd{};
                if constexpr (!LIFT) dd = *reinterpret_cast<const float4_t *>(sr + kRows + 8 * a);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 4 * (a & 3) + e;
                    const float y = LIFT ? S[a >> 2][i] * unit * P[a >> 2][i] : S[a >> 2][i] * (P[a >> 2][i] - dd[e]);
                    P[a >> 2][i] = !MASK || (seen >> i & 1u) ? y : 0.f;
                }
            }
            if constexpr (LIFT) {
                float t = 0.f;
#pragma unroll
                for (int n = 0; n < NSUB; ++n)
#pragma unroll
                    for (int i = 0; i < 16; ++i) t = fmaxf(t, fabsf(P[n][i]));
                if constexpr (LOOK) {
                    peak = fmaxf(peak, t);
                    return;
                }
                if (!CAREFUL && __any(t >= kMostDs)) {
                    const float f = lower(t);
#pragma unroll
                    for (int n = 0; n < NSUB; ++n) P[n] *= f;
                }
            }
            if constexpr (CAREFUL) {
                R::add_seen(ak, qt, ln, r0, P[0], seen);
            } else {
#pragma unroll
                for (int n = 0; n < NSUB; ++n) R::add(ak, qt, ln, r0 + 32 * n, P[n]);
            }
        };
        // One staged tile after the other, [x0, x1) of their order.
        auto each = [&](int x0, int x1, auto body) {
            for (int x = x0; x < x1; ++x) {
                staged_barrier();
                if (x + 1 < tiles) load(x + 1);
                if (busy) body(x, first_token(x));
                if (x + 1 < tiles) put(x + 1);
            }
        };
        if (tiles) {
            load(0);
            put(0);
        }
        // 32 rows of which none sees a key of the wave are left out
        auto left_out = [&](int t0, int r0) {
            const int a = t0 + (r0 ? half : 0), b = min(t0 + (r0 ? sh.tokens : half_end), tb) - 1;
            return r0 >= rows || a >= tb || k0 > b + shift || (k0 + 31 <= a + shift - W && k0 >= sh.sinks);
        };
        using std::integral_constant;
        if constexpr (CAREFUL) {
            each(0, tiles, [&](int x, int t0) {
                const bool all = x < whole;        // of such a tile 64 rows have one largest dS
#pragma unroll 1
                for (int r0 = 0; r0 < kRows; r0 += 32) {
                    if (left_out(t0, r0)) continue;
                    if constexpr (LIFT && MAKE_K) {
                        peak = 0.f;
#pragma unroll 1
                        for (int r = all ? 0 : r0; r < (all ? rows : r0 + 32); r += 32)
                            process(integral_constant<int, 1>{}, std::true_type{}, std::true_type{}, x, t0, r);
                        if (__any(peak >= kMostDs)) lower(peak);
                    }
                    process(integral_constant<int, 1>{}, std::true_type{}, std::false_type{}, x, t0, r0);
                }
            });
        } else {
            each(0, whole, [&](int x, int t0) {
                process(integral_constant<int, kRows / 32>{}, std::false_type{}, std::false_type{}, x, t0, 0);
            });
            each(whole, tiles, [&](int x, int t0) {
#pragma unroll 1
                for (int r0 = 0; r0 < kRows; r0 += 32)
                    if (!left_out(t0, r0))
                        process(integral_constant<int, 1>{}, std::true_type{}, std::false_type{}, x, t0, r0);
            });
        }
    };
    auto run = [&](auto make_v, auto make_k) {
        constexpr bool MAKE_V = decltype(make_v)::value, MAKE_K = decltype(make_k)::value;
        f32x16_t av[R::ND], ak[R::ND];
        walk(std::false_type{}, make_v, make_k, av, ak);
        bool bad = false;
        if constexpr (MAKE_V) bad |= any_not_finite(av);
        if constexpr (MAKE_K) bad |= any_not_finite(ak);
        bad &= part < 0 || key < sh.sinks;        // other keys' sums are dropped
        if (__syncthreads_or(busy && bad)) walk(std::true_type{}, make_v, make_k, av, ak);
        if (!busy) return;
        const float scale = LIFT ? sh.scale * inverse_power(unit * power_of_2(lift)) : sh.scale;
        const bool shared = fp.parts > 0 && jt == 0 && key < sh.sinks;   // the parts are added later
        if (part < 0) {
            const bool on = key < u.Lk && !shared;
            if (MAKE_K) store_column<T, D>(dk + at * D, ak, scale, on);
            if (MAKE_V) store_column<T, D>(dv + at * D, av, UNLIFT, on);
        }
        if (fp.parts > 0 && k0 < sh.sinks && jt == 0) {
            const int64_t slot = far_first(u.k0, far) + (part >= 0 ? part + 1 : 0);
            float *to = share + ((slot * sh.KV + u.hk) * 2 * sh.sinks + key) * (int64_t)D;
            if (MAKE_K) store_column<float, D>(to, ak, scale, shared && key < u.Lk);
            if (MAKE_V) store_column<float, D>(to + (int64_t)sh.sinks * D, av, UNLIFT, shared && key < u.Lk);
        }
    };
    if constexpr (kSplitKeySide<T, D>) {
        if (u.role == 0) run(std::true_type{}, std::false_type{});
        else run(std::false_type{}, std::true_type{});
    } else {
        run(std::true_type{}, std::true_type{});
    }
}

// Adds the parts' shares of the sinks' gradients: 32 neighbouring elements by 32 groups
// of lanes, which take the parts in turn and join in LDS, in a fixed order.
constexpr int kSinkLanes = 32;
template <typename T>
__global__ __launch_bounds__(1024) void swa_sinks_kernel(SwaShape sh, int pairs, int far, int D,
                                                         const float *__restrict__ share, T *__restrict__ dk,
                                                         T *__restrict__ dv) {
    __shared__ float sum[32][kSinkLanes + 1];
    if (sh.cu && sh.meta[1]) return;
    const int pair = (int)(blockIdx.z << kGridBits | blockIdx.x);   // sequence, key head
    if (pair >= pairs) return;
    const int n = pair / sh.KV, hk = pair - n * sh.KV;
    int64_t k0 = (int64_t)n * sh.Tk;
    int Lq = sh.T, Lk = sh.Tk;
    if (sh.cu) {
        Lq = sh.cu[n + 1] - sh.cu[n];
        k0 = sh.cuk[n], Lk = sh.cuk[n + 1] - sh.cuk[n];
    }
    const FarParts fp = far_parts(Lq, Lk, sh.window, sh.sinks, far);
    if (fp.parts == 0) return;
    // dK's elements, then dV's; D is a multiple of 32, so a block has one of them
    const int x = threadIdx.x % kSinkLanes, g = threadIdx.x / kSinkLanes, all = sh.sinks * D;
    const int i = blockIdx.y * kSinkLanes + x, e = i < all ? i : i - all;
    const int64_t step = (int64_t)sh.KV * 2 * all;
    const float *from = share + far_first(k0, far) * step + (int64_t)hk * 2 * all + i;
    const bool on = e / D < Lk;
    float a = 0.f;
    if (on)
#pragma unroll 4
        for (int p = g; p <= fp.parts; p += 32) a += from[p * step];
    sum[g][x] = a;
    __syncthreads();
    if (g || !on) return;
    a = 0.f;
#pragma unroll
    for (int p = 0; p < 32; ++p) a += sum[p][x];
    T *to = i < all ? dk : dv;
    to[((k0 + e / D) * sh.KV + hk) * D + e % D] = round_to<T>(a);
}

hipError_t launch_swa_bwd(const SwaArgs &a, hipStream_t st) {
    const SwaWorkspace w = swa_workspace_layout(a, true);
    const int rows = swa_row_tile(a), G = a.H / a.KV, far = swa_far_chunk(a.window);
    char *ws = static_cast<char *>(a.workspace);
    float *dsum = reinterpret_cast<float *>(ws + w.off_dsum), *share = reinterpret_cast<float *>(ws + w.off_far);
    SwaShape s{};
    s.T = a.T, s.Tk = a.Tk, s.H = a.H, s.KV = a.KV, s.G = G, s.window = a.window, s.sinks = a.sinks;
    s.tokens = rows / G;
    s.scale = a.scale, s.c = a.scale * 1.4426950408889634f;
    SwaShape sk = s;
    sk.tokens = kRows / G;
    int64_t units = w.row_units, key_units = w.key_units;
    bool join = a.sinks && (int64_t)a.Tk >= (int64_t)kSwaKeyTile + a.window;
    if (a.cu) {
        int32_t *meta = static_cast<int32_t *>(a.workspace);
        int2 *table = reinterpret_cast<int2 *>(ws + w.off_rows), *keys = reinterpret_cast<int2 *>(ws + w.off_keys);
        hipError_t e = launch_swa_table(a, true, s.tokens, meta, table, keys, st);
        if (e != hipSuccess) return e;
        s.cu = sk.cu = a.cu, s.cuk = sk.cuk = a.cuk;
        s.meta = meta, s.table = table;
        sk.meta = meta + 2, sk.table = keys;
    } else {
        const FarParts fp = far_parts(a.T, a.Tk, a.window, a.sinks, far);
        s.per_seq = (a.T + s.tokens - 1) / s.tokens;
        sk.per_seq = (a.Tk + kSwaKeyTile - 1) / kSwaKeyTile + fp.parts;
        units = (int64_t)s.per_seq * a.N;
        key_units = (int64_t)sk.per_seq * a.N;
        s.units = (int)units, sk.units = (int)key_units;
        join = fp.parts > 0;
    }
    return swa_with<false>(a.dtype, a.D, [&](auto t, auto dim) {
        using T = decltype(t);
        constexpr int D = decltype(dim)::value, RB = Rows<T, D>::RB;
        auto in = [](const void *p) { return static_cast<const T *>(p); };
        auto out = [](void *p) { return static_cast<T *>(p); };
        hipError_t e = hipSuccess;
        if (units) {
            ProfScope prof("gdn_swa_dq", st);
            auto go = [&](auto waves) {
                constexpr int NW = decltype(waves)::value, lds = 4 * kKeys * RB;
                hipError_t x = swa_lds(swa_dq_kernel<T, D, NW>, lds);
                if (x != hipSuccess) return x;
                swa_dq_kernel<T, D, NW><<<swa_grid(units * a.KV), 64 * NW, lds, st>>>(
                    s, in(a.q), in(a.k), in(a.v), in(a.o), a.lse, in(a.d_o), out(a.dq), dsum);
                return hipGetLastError();
            };
            e = rows == 64 ? go(std::integral_constant<int, 2>{}) : go(std::integral_constant<int, 4>{});
            if (e != hipSuccess) return e;
        }
        if (key_units) {
            ProfScope prof("gdn_swa_dkv", st);
            constexpr int lds = 4 * kRows * RB + 5 * kRows * 4;
            e = swa_lds(swa_dkv_kernel<T, D>, lds);
            if (e != hipSuccess) return e;
            constexpr int roles = kSplitKeySide<T, D> ? 2 : 1;
            swa_dkv_kernel<T, D><<<swa_grid(key_units * a.KV * roles), 256, lds, st>>>(
                sk, far, in(a.q), in(a.k), in(a.v), a.lse, in(a.d_o), dsum, out(a.dk), out(a.dv), share);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        if (join) {
            ProfScope prof("gdn_swa_sinks", st);
            const int pairs = a.N * a.KV;
            const dim3 all = swa_grid(pairs), grid(all.x, (unsigned)(2 * a.sinks * D / kSinkLanes), all.y);
            swa_sinks_kernel<T><<<grid, 1024, 0, st>>>(s, pairs, far, D, share, out(a.dk), out(a.dv));
            e = hipGetLastError();
        }
        return e;
    });
}

}  // namespace gdn
