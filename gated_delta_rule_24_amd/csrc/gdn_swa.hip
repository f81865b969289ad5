// Windowed attention with sinks, forward:
//   query at position p sees key j iff j <= p and (p - j < window or j < sinks)
//   o = sum_j exp(s_j - lse) v_j,  s_j = scale q k_j,  lse = log sum_j exp(s_j)
// over the visible keys, in one pass with the running maximum and sum of the
// softmax in fp32.
//
// A wave owns 32 rows (query token, head of the group).  It forms S^T = K Q^T in
// 32 x 32 matrix-core tiles, so that a lane holds one row's scores: the maximum
// and sum over keys stay in the lane but for one exchange of the wave's halves,
// and the probabilities are, as they lie, the operand of O^T += V^T P^T (K rows by
// 16-byte LDS reads, V by transposing ones).  Q and O^T stay in registers.  The
// waves of a block share tiles of 64 keys, copied straight to LDS one tile ahead.
// Only tiles that the mask cuts are masked; tiles that it hides are not visited.
//
// Measured (MI355X; a bf16 8192^3 product 1.23 PFLOP/s, a copy 5.35 TB/s): 50408 packed
// tokens, 16 heads of 128, window 2048, bf16: 810 to 865 us from one GPU to another, 0.85
// PFLOP/s of visible pairs; fp16 905 to 935.  The matrix cores are busy 42% of the time and the vector units about as
// long (per 64 keys and wave 32 products of 32 cycles, 127 vector instructions, 32
// exponentials of 16 cycles): two waves a SIMD, all that the registers allow, overlap
// the two in part.  Reads of LDS meet no bank twice (before the swizzle of gdn_swa.h:
// 1245 us instead of 966).  256 sequences of 9 tokens behind 2052 keys: 202 us, 5.4 TB/s.
// In fp32 6.84 ms (0.104 PFLOP/s of 0.14), 64-wide heads 3.11; 256-wide heads 2.04 ms in bf16
// (0.70 PFLOP/s), 2.16 in fp16.  These hold 512 bytes and more of a row in several forms
// and run one wave a SIMD: with two they spill, 7.53 ms in fp32 (128) and 3.84 in bf16 (256).
// Tried and not kept: tiles of 32 keys (885 us instead of 835; three waves a SIMD
// spill), raised wave priority in the products (845 to 850 instead of 839).
#include "gdn_ops.h"
#include "gdn_swa.h"

#include <algorithm>

namespace gdn {

constexpr int kKeys = 64;            // keys of a staged tile
// log2: how far scores may pass the maximum that is subtracted.  Probabilities are
// taken times 2^kLift: in fp16 the small ones, which many keys may share, would be
// subnormal or 0.  Their sum has the same factor.  The two fill fp16's range (2^15.9 <
// 65504), and of the two the lift keeps bits: probabilities down to 2^-28 of the
// largest have all of theirs, for 3% more time (50408 packed tokens, 16 heads of 128, fp16:
// 922 us, 897 with a slack of 8).
template <typename T>
constexpr float kSlack = std::is_same_v<T, _Float16> ? 0.9f : 8.f;
template <typename T>
constexpr float kLift = std::is_same_v<T, _Float16> ? 15.f : 0.f;
constexpr float kFarScores = 0x1p18f;   // log2: past this a maximum's rounding is no longer a small power

template <typename T, int D, int NW>
__global__ __launch_bounds__(64 * NW, (Rows<T, D>::RB >= 512 ? 1 : 2)) void swa_fwd_kernel(SwaShape sh, const T *__restrict__ q,
                                                                          const T *__restrict__ k,
                                                                          const T *__restrict__ v, T *__restrict__ o,
                                                                          float *__restrict__ lse) {
    using R = Rows<T, D>;
    constexpr int RB = R::RB, TILE = kKeys * RB, PIECES = TILE / 1024 / NW;
    extern __shared__ __align__(16) char smem[];   // two stages of K and V tiles
    SwaUnit u;
    if (!swa_find(sh, true, u)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, h = l >> 5;
    const int shift = u.Lk - u.Lq;                 // position of a token less its index
    const int t0 = u.unit * sh.tokens, t1 = min(t0 + sh.tokens, u.Lq);   // the block's tokens
    const int pfirst = t0 + shift, plast = t1 - 1 + shift;
    const int W = sh.window;

    // the wave's and the lane's rows
    const int row = wave * 32 + (l & 31), tt = row / sh.G, token = t0 + tt;
    const bool on = tt < sh.tokens && token < t1;
    const int pos = min(token, t1 - 1) + shift;
    const int w0 = t0 + wave * 32 / sh.G;
    const bool busy = w0 < t1 && wave * 32 / sh.G < sh.tokens;
    const int p0 = w0 + shift, p1 = min(t0 + (wave * 32 + 31) / sh.G, t1 - 1) + shift;
    const int64_t at = (u.q0 + min(token, t1 - 1)) * sh.H + u.hk * sh.G + row % sh.G;
    u32x4_t qf[R::NS];
#pragma unroll
    for (int s = 0; s < R::NS; ++s)
        qf[s] = *reinterpret_cast<const u32x4_t *>(reinterpret_cast<const char *>(q + at * D) + 32 * s + 16 * h);
#pragma unroll
    for (int s = 0; s < R::NS; ++s) arrived(qf[s]);

    // key tiles: the sinks, then the band from `low`; one range where they meet
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
    float m, sum;                                  // log2 of what sums count in; this lane's part of the sum
    bool far = false;                              // m is the largest score itself, subtracted before the scale
    const typename R::Lane lane;
    // All tiles.  CAREFUL: what a row does not see may be infinite or NaN, and scores may
    // be so large that the maximum less its rounding is far from 0.  That is seen from
    // sums that are not finite and from the maximum, and all is done again: it keeps the
    // rare path's registers and its looks at V out of the other.  It takes the same steps, 32
    // keys at a time: rows that see nothing of the kind come out with the same bits.
    auto walk = [&](auto careful) {
        constexpr bool CAREFUL = decltype(careful)::value;
#pragma unroll
        for (int dt = 0; dt < R::ND; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[dt][i] = 0.f;
        m = -__builtin_inff(), sum = 0.f;
        // One staged tile after the other, [x0, x1) of their order.
        auto each = [&](int x0, int x1, auto body) {
            for (int x = x0; x < x1; ++x) {
                staged_barrier();
                if (x + 1 < tiles) load(x + 1);
                if (busy) body(tile_at(x), smem + (x & 1) * 2 * TILE);
            }
        };
        // A row's maximum follows a tile's largest score.  That is the row's own matter: no bit
        // of its sums comes from the wave's other rows.
        auto raise = [&](float top) {
            // the largest exponent as it is taken below, so that no rounding of m adds to it
            const bool over = CAREFUL && far ? top > m : fmaf(top, sh.c, -m) > kLift<T> + kSlack<T>;
            if (__any(over)) {
                const float up = !over ? m : CAREFUL && far ? top : fmaf(top, sh.c, -kLift<T>);
                const float f = over ? __builtin_amdgcn_exp2f((m - up) * (CAREFUL && far ? sh.c : 1.f)) : 1.f;
                m = up;
                sum *= f;
#pragma unroll
                for (int dt = 0; dt < R::ND; ++dt)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[dt][i] *= f;
            }
        };
        // Scores of the 32 keys from j0 + r0 on: -inf where the row does not see them.
        auto mask = [&](f32x16_t &S, int j0, int jend, int r0, const typename R::Lane &ln) {
            uint32_t seen = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int j = j0 + r0 + 4 * (ln.l >> 5) + 8 * (i >> 2) + (i & 3);
                const bool see = j <= pos && j < jend && (j > pos - W || j < sh.sinks);
                S[i] = see ? S[i] : -__builtin_inff();
                seen |= (uint32_t)see << i;
            }
            return seen;
        };
        auto largest = [](float top, const f32x16_t &S) {
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, S[i]);
            return top;
        };
        auto process = [&](auto subs, auto masked, const char *kt, int j0, int jend, int r0) {
            const char *vt = kt + TILE;
            constexpr int NSUB = decltype(subs)::value;
            constexpr bool MASK = decltype(masked)::value;
            const typename R::Lane ln = lane.fresh();
            f32x16_t S[NSUB];
#pragma unroll
            for (int n = 0; n < NSUB; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) S[n][i] = 0.f;
            R::dot(S, kt, ln, r0, qf);
            uint32_t seen = 0;
            if constexpr (MASK) seen = mask(S[0], j0, jend, r0, ln);
            if constexpr (!CAREFUL) {
                float top = S[0][0];
#pragma unroll
                for (int n = 0; n < NSUB; ++n) top = largest(top, S[n]);
                raise(half_max(top));
            }
            const float base = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
            for (int n = 0; n < NSUB; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = CAREFUL && far ? fmaf(S[n][i] - base, sh.c, kLift<T>) : fmaf(S[n][i], sh.c, -base);
                    S[n][i] = __builtin_amdgcn_exp2f(x);
                    sum += S[n][i];
                }
            if constexpr (CAREFUL) {
                R::add_seen(acc, vt, ln, r0, S[0], seen);
                return;
            }
#pragma unroll
            for (int n = 0; n < NSUB; ++n) R::add(acc, vt, ln, r0 + 32 * n, S[n]);
            if constexpr (!MASK && !R::F32) reads_ahead<2, NSUB * 2 * R::ND, 4>();
        };
        using std::integral_constant;
        if (tiles) load(0);
        // 32 keys that no row of the wave sees are left out
        auto left_out = [&](int j, int jend) { return j > p1 || j >= jend || (j + 31 <= p0 - W && j >= sh.sinks); };
        if constexpr (CAREFUL) {
            int x = 0;
            each(0, tiles, [&](int it, const char *kt) {
                const bool all = x++ < whole;      // of such a tile 64 keys have one maximum
                const int j0 = first_key(it), jend = it < ns ? sh.sinks : high;
#pragma unroll 1
                for (int r0 = 0; r0 < kKeys; r0 += 32) {
                    if (left_out(j0 + r0, jend)) continue;
                    float top = -__builtin_inff();
#pragma unroll 1
                    for (int r = all ? 0 : r0; r < (all ? kKeys : r0 + 32); r += 32) {
                        const typename R::Lane ln = lane.fresh();
                        f32x16_t S[1];
#pragma unroll
                        for (int i = 0; i < 16; ++i) S[0][i] = 0.f;
                        R::dot(S, kt, ln, r, qf);
                        mask(S[0], j0, jend, r, ln);
                        top = largest(top, S[0]);
                    }
                    raise(half_max(top));
                    process(integral_constant<int, 1>{}, std::true_type{}, kt, j0, jend, r0);
                }
            });
        } else {
            each(0, whole, [&](int it, const char *kt) {
                process(integral_constant<int, kKeys / 32>{}, std::false_type{}, kt, first_key(it), 0, 0);
            });
            each(whole, tiles, [&](int it, const char *kt) {
                const int j0 = first_key(it), jend = it < ns ? sh.sinks : high;
#pragma unroll 1
                for (int r0 = 0; r0 < kKeys; r0 += 32)
                    if (!left_out(j0 + r0, jend)) process(integral_constant<int, 1>{}, std::true_type{}, kt, j0, jend, r0);
            });
        }
    };
    walk(std::false_type{});
    const bool large = fabsf(m) > kFarScores && fabsf(m) < __builtin_inff();
    far = __syncthreads_or(busy && large);
    const bool again = __syncthreads_or(busy && any_not_finite(acc)) || far;
    if (again) walk(std::true_type{});
    if (far) m = fmaf(m, sh.c, -kLift<T>);

    if (!busy) return;
    sum = half_sum(sum);
    if (again && sum == 0.f)                       // nothing but scores of -inf: no value counts
#pragma unroll
        for (int dt = 0; dt < R::ND; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[dt][i] = 0.f;
    store_column<T, D>(o + at * D, acc, sum == 0.f ? 0.f : 1.f / sum, on);
    if (lse && on && h == 0)
        lse[at] = sum == 0.f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
}

// ---- packed batches: the table of units ---------------------------------------------

// Block 0: the query tiles' table, block 1: the key tiles'.
__global__ __launch_bounds__(1024) void swa_table_kernel(int N, int T, int Tk, const int32_t *__restrict__ cu,
                                                         const int32_t *__restrict__ cuk, int tokens, int window,
                                                         int sinks, int far, int most_rows, int most_keys,
                                                         int32_t *__restrict__ meta, int2 *__restrict__ rows,
                                                         int2 *__restrict__ keys) {
    const bool key_side = blockIdx.x == 1;
    const int most = key_side ? most_keys : most_rows;
    int2 *table = key_side ? keys : rows;
    meta += 2 * blockIdx.x;
    __shared__ int first[1025], part[16], code;
    const int tid = threadIdx.x;
    if (tid == 0) code = 0;
    __syncthreads();
    int bad = 0;
    for (int n = tid; n < N; n += 1024) {
        if (cu[n + 1] < cu[n]) bad |= 2;
        if (cuk[n + 1] < cuk[n]) bad |= 16;
    }
    if (tid == 0) {
        if (cu[0] != 0) bad |= 1;
        if (cu[N] != T) bad |= 4;
        if (cuk[0] != 0) bad |= 8;
        if (cuk[N] != Tk) bad |= 32;
    }
    if (bad) atomicOr(&code, bad);
    __syncthreads();
    bad = code;
    int total = 0;
    for (int n0 = 0; n0 < N && !bad; n0 += 1024) {
        const int n = n0 + tid;
        int x = 0;
        if (n < N) {
            const int Lq = cu[n + 1] - cu[n], Lk = cuk[n + 1] - cuk[n];
            if (key_side) {
                x = (Lk + kSwaKeyTile - 1) / kSwaKeyTile;
                // tokens past those that the first key tile's window reaches
                const int64_t reach = (int64_t)kSwaKeyTile + window - 1 - (Lk - Lq);
                const int rest = (int)min((int64_t)Lq, max((int64_t)Lq - reach, (int64_t)0));
                if (x && sinks) x += (rest + far - 1) / far;
            } else {
                x = (Lq + tokens - 1) / tokens;
            }
        }
        int sum = x;
        for (int d = 1; d < 64; d <<= 1) {
            const int y = __shfl_up(sum, d, 64);
            if ((tid & 63) >= d) sum += y;
        }
        if ((tid & 63) == 63) part[tid >> 6] = sum;
        __syncthreads();
        for (int w = 0; w < (tid >> 6); ++w) sum += part[w];
        first[tid + 1] = sum;
        if (tid == 0) first[0] = 0;
        __syncthreads();
        const int here = first[1024];
        for (int i = tid; i < here && total + i < most; i += 1024) {
            int a = 0, b = 1024;                   // the last sequence whose first unit is at most i
            while (b - a > 1) {
                const int c = (a + b) / 2;
                if (first[c] <= i) a = c;
                else b = c;
            }
            table[total + i] = int2{n0 + a, i - first[a]};
        }
        total += here;
        __syncthreads();
    }
    if (tid == 0) {
        meta[0] = min(total, most);
        meta[1] = bad ? __builtin_ctz(bad) + 1 : 0;
    }
}

hipError_t launch_swa_table(const SwaArgs &a, bool bwd, int tokens, int32_t *meta, int2 *rows, int2 *keys,
                            hipStream_t st) {
    ProfScope prof("gdn_swa_table", st);
    const SwaWorkspace w = swa_workspace_layout(a, bwd);
    swa_table_kernel<<<bwd ? 2 : 1, 1024, 0, st>>>(a.N, a.T, a.Tk, a.cu, a.cuk, tokens, a.window, a.sinks,
                                                   swa_far_chunk(a.window), (int)w.row_units, (int)w.key_units, meta, rows,
                                                   keys);
    return hipGetLastError();
}

// Rows of a block's tile, 32 to a wave.  Half as many where that still leaves CUs without
// a block.  Measured with 128 and 64 rows, forward: 3 x 333 tokens, 6 heads on 2 of 64,
// window 100 (48 blocks) 13.0 and 11.5 us; 256 sequences of 9 tokens on 2061 keys, 16 heads
// on 4 of 128 (1324 blocks, a third of their rows used) 202 and 232 us; of 25 tokens 245
// and 297; 50408 packed tokens, 16 heads of 128, 860 and 1183 us.  dQ of 1237 tokens, 4 heads
// on 2 of 32 in fp32, 20.7 and 17.5 us.
int swa_row_tile(const SwaArgs &a) {
    const int64_t blocks = ((int64_t)a.B * a.T / (128 / (a.H / a.KV)) + a.N) * a.KV;
    return blocks < 256 ? 64 : 128;
}

SwaWorkspace swa_workspace_layout(const SwaArgs &a, bool bwd) {
    SwaWorkspace w{};
    const int tokens = swa_row_tile(a) / (a.H / a.KV);
    const int64_t T = (int64_t)a.B * a.T, Tk = (int64_t)a.B * a.Tk, far = swa_far_chunk(a.window);
    const bool table = a.B == 1;                  // a packed batch, or one sequence
    w.row_units = T / tokens + a.N;
    w.far_units = a.sinks ? Tk / far : 0;         // a sequence has keys / far at most
    w.key_units = Tk / kSwaKeyTile + a.N + w.far_units;
    size_t at = 256;
    auto take = [&](size_t bytes) {
        const size_t x = at;
        at += (bytes + 255) / 256 * 256;
        return x;
    };
    w.off_rows = take(table ? (size_t)w.row_units * 8 : 0);
    if (bwd) {
        w.off_keys = take(table ? (size_t)w.key_units * 8 : 0);
        w.off_dsum = take((size_t)T * a.H * 4);
        // every part of the sinks' tile, the near ones included: dK and dV of the sinks in fp32
        w.off_far = take((size_t)(2 * w.far_units) * a.KV * 2 * a.sinks * a.D * 4);
    }
    w.total = at;
    return w;
}

hipError_t launch_swa_fwd(const SwaArgs &a, hipStream_t st) {
    const SwaWorkspace w = swa_workspace_layout(a, false);
    const int rows = swa_row_tile(a), G = a.H / a.KV;
    SwaShape s{};
    s.T = a.T, s.Tk = a.Tk, s.H = a.H, s.KV = a.KV, s.G = G, s.window = a.window, s.sinks = a.sinks;
    s.tokens = rows / G;
    s.scale = a.scale, s.c = a.scale * 1.4426950408889634f;
    int64_t units = w.row_units;
    if (a.cu) {
        int32_t *meta = static_cast<int32_t *>(a.workspace);
        int2 *table = reinterpret_cast<int2 *>(static_cast<char *>(a.workspace) + w.off_rows);
        hipError_t e = launch_swa_table(a, false, s.tokens, meta, table, nullptr, st);
        if (e != hipSuccess) return e;
        s.cu = a.cu, s.cuk = a.cuk, s.meta = meta, s.table = table;
    } else {
        s.per_seq = (a.T + s.tokens - 1) / s.tokens;
        units = (int64_t)s.per_seq * a.N;
        s.units = (int)units;
    }
    if (units == 0) return hipSuccess;
    ProfScope prof("gdn_swa_fwd", st);
    return swa_with<true>(a.dtype, a.D, [&](auto t, auto dim) {
        using T = decltype(t);
        constexpr int D = decltype(dim)::value;
        auto go = [&](auto waves) {
            constexpr int NW = decltype(waves)::value;
            constexpr int lds = 4 * kKeys * Rows<T, D>::RB;
            hipError_t e = swa_lds(swa_fwd_kernel<T, D, NW>, lds);
            if (e != hipSuccess) return e;
            swa_fwd_kernel<T, D, NW><<<swa_grid(units * a.KV), 64 * NW, lds, st>>>(
                s, static_cast<const T *>(a.q), static_cast<const T *>(a.k), static_cast<const T *>(a.v),
                static_cast<T *>(a.o), a.lse);
            return hipGetLastError();
        };
        return rows == 64 ? go(std::integral_constant<int, 2>{}) : go(std::integral_constant<int, 4>{});
    });
}

}  // namespace gdn
