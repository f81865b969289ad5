// Shared parts of windowed attention (gdn_swa.hip forward, gdn_swa_bwd.hip
// gradient): the call's shape, which unit of work a block has, and products
// of 32 x 32 tiles whose operands lie in LDS as rows.
//
// The query heads that share a key head are rows of one matrix: row r of a tile
// is query token r / G, head r mod G of the group (G = heads / kv_heads), so
// keys and values are staged once for the group, and a few tokens of many
// heads fill a tile.  A tile takes whole tokens (rows / G of them); what is
// left over of its rows is computed and dropped.
#pragma once

#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_types.h"

namespace gdn {

constexpr int kSwaMaxGroup = 16;
constexpr int kSwaMaxSinks = 128;
constexpr int kSwaKeyTile = 128;     // keys of a block of the key gradient

struct SwaArgs {
    int32_t B, T, Tk, N, H, KV, D, window, sinks, dtype;
    float scale;
    const void *q, *k, *v;
    const int32_t *cu, *cuk;         // packed, or both NULL
    void *o;                         // forward: written
    float *lse;
    const void *d_o;                 // backward
    void *dq, *dk, *dv;
    void *workspace;
};

// Workspace (byte offsets): status words and the table of units (packed), then
// for the backward pass D = rowsum(dO o), the far parts' share of the sinks'
// gradients, and its own tables.
struct SwaWorkspace {
    int64_t row_units, key_units, far_units;   // upper bounds
    size_t off_rows, off_keys, off_dsum, off_far;
    size_t total;
};
int swa_row_tile(const SwaArgs &a);
SwaWorkspace swa_workspace_layout(const SwaArgs &a, bool bwd);
hipError_t launch_swa_fwd(const SwaArgs &a, hipStream_t stream);
hipError_t launch_swa_bwd(const SwaArgs &a, hipStream_t stream);

// Tokens of far queries in one part of the sinks' key gradient: as many as the near
// part of a key tile has.
inline int swa_far_chunk(int window) { return window + kSwaKeyTile; }

// Builds the tables of units of a packed batch, int2 {sequence, unit of the
// sequence}: tiles of `tokens` query tokens, and for the backward pass the far
// parts of the sinks and then the key tiles.  meta: {units of
// the first table, code of the offsets' check, units of the second, the code}.
hipError_t launch_swa_table(const SwaArgs &a, bool bwd, int tokens, int32_t *meta, int2 *rows, int2 *keys,
                            hipStream_t stream);

// What the kernels need to find a block's unit.
struct SwaShape {
    int32_t T, Tk, H, KV, G, window, sinks;
    int32_t tokens;                  // query tokens of a tile
    int32_t per_seq;                 // units of a sequence (not packed)
    int32_t units;                   // of all sequences (not packed)
    const int32_t *cu, *cuk, *meta;  // packed
    const int2 *table;
    float c;                         // scale log2(e)
    float scale;
};

// A launch counts its threads along x in 32 bits: blocks past 2^20 go on along y.
constexpr int kGridBits = 20;
inline dim3 swa_grid(int64_t blocks) {
    blocks = (blocks + 7) / 8 * 8;
    if (blocks <= 1 << kGridBits) return dim3((unsigned)blocks);
    return dim3(1u << kGridBits, (unsigned)((blocks + (1 << kGridBits) - 1) >> kGridBits));
}

struct SwaUnit {
    int unit, hk, role;              // unit of the sequence, key head, which of `roles`
    int64_t q0, k0;                  // the sequence's first query and key
    int Lq, Lk, n;
};

// The unit of this block; false: none.  Blocks go to the 8 XCDs in turn: each
// XCD takes a contiguous share of the units, neighbouring tiles of one head, so
// that the keys that they share are in one L2.  last_first: in falling order, as
// later queries see more keys and the longest units should begin first.  ROLES
// blocks in a row have the same unit, each another part of its work.
template <int ROLES = 1>
__device__ __forceinline__ bool swa_find(const SwaShape &s, bool last_first, SwaUnit &u) {
    int units = s.units;
    if (s.cu) {
        if (s.meta[1]) return false;
        units = s.meta[0];
    }
    const int64_t total = (int64_t)units * s.KV * ROLES;
    const uint32_t block = blockIdx.y << kGridBits | blockIdx.x;
    const int64_t per = (total + 7) / 8, i = block >> 3;
    int64_t at = (block & 7) * per + i;
    if (i >= per || at >= total) return false;
    const int pairs = s.cu ? 0 : units / max(s.per_seq, 1) * s.KV;
    if (pairs % 8 == 0 && !s.cu) {   // whole (sequence, key head) pairs to an XCD: the longest units of all of them first
        const int share = pairs / 8 * ROLES;
        const int x = (int)(i / share), y = (int)(i - (int64_t)x * share);
        const int pair = (block & 7) * (pairs / 8) + y / ROLES;
        u.role = y % ROLES;
        u.hk = pair % s.KV;
        u.n = pair / s.KV;
        u.unit = last_first ? s.per_seq - 1 - x : x;
        u.q0 = (int64_t)u.n * s.T, u.Lq = s.T;
        u.k0 = (int64_t)u.n * s.Tk, u.Lk = s.Tk;
        return true;
    }
    u.role = (int)(at % ROLES);
    at /= ROLES;
    u.hk = (int)(at / units);
    const int y = (int)(at - (int64_t)u.hk * units), x = last_first ? units - 1 - y : y;
    if (s.cu) {
        const int2 e = s.table[x];
        u.n = e.x;
        u.unit = e.y;
        const int q0 = s.cu[e.x], k0 = s.cuk[e.x];
        u.q0 = q0, u.Lq = s.cu[e.x + 1] - q0;
        u.k0 = k0, u.Lk = s.cuk[e.x + 1] - k0;
    } else {
        u.n = x / s.per_seq;
        u.unit = x - u.n * s.per_seq;
        u.q0 = (int64_t)u.n * s.T, u.Lq = s.T;
        u.k0 = (int64_t)u.n * s.Tk, u.Lk = s.Tk;
    }
    return true;
}

// ---- tiles in LDS --------------------------------------------------------------

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// acc += A B over one 16-byte chunk of both operands' rows.  32 x 32 tiles:
// lane l, m = l % 32, h = l / 32.  The accumulator holds C[8 (i / 4) + 4 h + i % 4][m]
// in element i < 16; a lane supplies row m of A and column m of B, the two halves
// h different chunks.
template <typename T>
__device__ __forceinline__ void mma32(f32x16_t &acc, u32x4_t a, u32x4_t b) {
    if constexpr (std::is_same_v<T, bf16_t>) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                     __builtin_bit_cast(bf16x8_t, b), acc, 0, 0, 0);
    } else if constexpr (std::is_same_v<T, _Float16>) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b),
                                                    acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i]), __uint_as_float(b[i]), acc, 0, 0, 0);
    }
}

// Two fp32 values as 16-bit values in one word, rounded to nearest.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (std::is_same_v<T, bf16_t>) {
        return pack_bf16x2(a, b);
    } else {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        typedef float f2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), h2));
    }
}

__device__ __forceinline__ uint32_t lds_addr(const void *p) { return (uint32_t)(uintptr_t)p; }

// Rows of D elements in LDS, each RB bytes, their 16-byte chunks permuted by the
// row.  Of the 256 bytes across the banks the chunk (row, c) takes c ^ swz(row) (and
// a place by the row where several fit): sixteen rows at one chunk meet no bank
// twice, and neither do the four rows by 64 bytes of half a transposing read.
template <typename T, int D>
struct Rows {
    static constexpr int RB = D * (int)sizeof(T);
    static constexpr int NS = RB / 32;                    // chunk pairs, steps of a product over D
    static constexpr int RPL = RB >= 256 ? 1 : 256 / RB;  // rows across the banks
    static constexpr int ND = D / 32;                     // tiles along D
    static constexpr bool F32 = std::is_same_v<T, float>;
    __device__ __forceinline__ static int swz(int row) {  // swz(row + 8) = swz(row) ^ 2, swz(row + 16) = swz(row)
        const int x = row / RPL;
        return RPL == 1 ? (x & 3) << 2 | (x >> 2 & 3) : RPL == 2 ? (x & 1) << 2 | (x >> 1 & 3) : x & 3;
    }
    __device__ __forceinline__ static int chunk_off(int row, int chunk) { return row * RB + ((chunk ^ swz(row)) << 4); }
    // The chunk that lies at byte b of a tile.
    __device__ __forceinline__ static int chunk_at(int b) { return (b % RB / 16) ^ swz(b / RB); }
    // What a lane's reads start from.  fresh(): the same values, which the compiler
    // takes for new ones, so that it forms addresses where they are used instead of
    // keeping all of them in registers.
    struct Lane {
        int l, row, col;
        __device__ __forceinline__ Lane() {
            l = threadIdx.x & 63;
            row = chunk_off(l & 31, l >> 5);
            const int s = l & 15;
            col = chunk_off(4 * (l >> 5) + (s >> 2), 2 * (l >> 4 & 1) + (s >> 1 & 1)) + ((s & 1) << 3);
        }
        __device__ __forceinline__ Lane fresh() const {
            Lane x = *this;
            asm volatile("" : "+v"(x.l), "+v"(x.row), "+v"(x.col));
            return x;
        }
    };
    // Operand rows r0 .. r0 + 31 (r0 a multiple of 32), step s of the product over D.
    __device__ __forceinline__ static u32x4_t frag(const char *t, const Lane &ln, int r0, int s) {
        return *reinterpret_cast<const u32x4_t *>(t + (ln.row ^ (s << 5)) + r0 * RB);
    }
    // S[n] += the product over D of rows r0 + 32 n .. +31 with the operand b, N tiles side by
    // side.  The reads go in batches, each ahead of the products of the one before it:
    // left to itself the compiler puts a read right in front of its product.
    template <int N>
    __device__ __forceinline__ static void dot(f32x16_t (&S)[N], const char *t, const Lane &ln, int r0,
                                               const u32x4_t (&b)[NS]) {
        constexpr int ALL = N * NS, BATCH = F32 ? 2 : 8;
        auto read = [&](int i) { return frag(t, ln, r0 + 32 * (i % N), i / N); };
        u32x4_t f[2][BATCH];
#pragma unroll
        for (int i = 0; i < BATCH && i < ALL; ++i) f[0][i] = read(i);
#pragma unroll
        for (int i0 = 0; i0 < ALL; i0 += BATCH) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < BATCH && i0 + BATCH + i < ALL; ++i) f[(i0 / BATCH + 1) & 1][i] = read(i0 + BATCH + i);
#pragma unroll
            for (int i = 0; i < BATCH && i0 + i < ALL; ++i)
                mma32<T>(S[(i0 + i) % N], f[(i0 / BATCH) & 1][i], b[(i0 + i) / N]);
        }
    }
    // Columns 32 dt .. +31 of rows r0 .. r0 + 31 as the A operand of a product
    // over the rows, in the order in which an accumulator holds its rows.
    // 16 bits: rows 16 ks .. +15 of them.
    __device__ __forceinline__ static u32x4_t col16(const char *t, const Lane &ln, int r0, int ks, int dt) {
        const char *p = t + (r0 + 16 * ks) * RB;
        const uint2 lo = lds_read_tr16(p + (ln.col ^ (dt << 6))), hi = lds_read_tr16(p + (ln.col ^ (dt << 6) ^ 32) + 8 * RB);
        return u32x4_t{lo.x, lo.y, hi.x, hi.y};
    }
    // fp32: the lane's value of the row that accumulator element i stands for.
    __device__ __forceinline__ static float col32(const char *t, const Lane &ln, int r0, int i, int dt) {
        const int m = ln.l & 31;
        return *reinterpret_cast<const float *>(
            t + chunk_off(4 * (ln.l >> 5) + (i & 3) + 8 * (i >> 2), 8 * dt + (m >> 2)) + 4 * (m & 3) + r0 * RB);
    }

    // acc[dt] += X^T W: rows r0 .. r0 + 31 of X, W in the accumulator layout of a
    // 32 x 32 tile (rounded to T, to nearest, as an operand).
    __device__ __forceinline__ static void add(f32x16_t (&acc)[ND], const char *t, const Lane &ln, int r0,
                                               const f32x16_t &w) {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int dt = 0; dt < ND; ++dt)
                    acc[dt] = __builtin_amdgcn_mfma_f32_32x32x2f32(col32(t, ln, r0, i, dt), w[i], acc[dt], 0, 0, 0);
        } else {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                u32x4_t b;
#pragma unroll
                for (int e = 0; e < 4; ++e) b[e] = pack2<T>(w[8 * ks + 2 * e], w[8 * ks + 2 * e + 1]);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) mma32<T>(acc[dt], col16(t, ln, r0, ks, dt), b);
            }
        }
    }

    // add() for a tile that hides some of its (row, column) pairs and whose rows
    // may not be finite: a hidden pair has weight 0, and 0 times infinity must
    // not count.  The rows' finite values go through add()'s product.  What is seen
    // of +inf and NaN then adds a product that overflows to +inf, what is seen of
    // -inf and NaN one to -inf: both make a NaN, and a hidden one adds 0.  seen: bit
    // i for accumulator element i.
    __device__ __forceinline__ static void add_seen(f32x16_t (&acc)[ND], const char *t, const Lane &ln, int r0,
                                                    const f32x16_t &w, uint32_t seen) {
        constexpr float BIG = 0x1p127f;
        auto finite = [](float x) { return fabsf(x) < __builtin_inff() ? x : 0.f; };
        auto large = [](float x, float sign) {        // sign BIG where x is NaN or the infinity of that sign
            return !(fabsf(x) < __builtin_inff()) && !(x * sign < 0.f) ? sign * BIG : 0.f;
        };
        const f32x16_t zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int dt = 0; dt < ND; ++dt)
                    acc[dt] = __builtin_amdgcn_mfma_f32_32x32x2f32(finite(col32(t, ln, r0, i, dt)), w[i], acc[dt], 0, 0, 0);
#pragma unroll 1
            for (float sign = 1.f; sign >= -1.f; sign -= 2.f)
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) {
                    f32x16_t z = zero;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        z = __builtin_amdgcn_mfma_f32_32x32x2f32(large(col32(t, ln, r0, i, dt), sign),
                                                                 seen >> i & 1u ? BIG : 0.f, z, 0, 0, 0);
                    acc[dt] += z;
                }
        } else {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                u32x4_t b;
#pragma unroll
                for (int e = 0; e < 4; ++e) b[e] = pack2<T>(w[8 * ks + 2 * e], w[8 * ks + 2 * e + 1]);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) {
                    u32x4_t a = col16(t, ln, r0, ks, dt);
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[e] = pack2<T>(finite(half_of(a[e])), finite(half_of(a[e] >> 16)));
                    mma32<T>(acc[dt], a, b);
                }
            }
#pragma unroll 1
            for (float sign = 1.f; sign >= -1.f; sign -= 2.f)
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) {
                    f32x16_t z = zero;
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        u32x4_t a = col16(t, ln, r0, ks, dt), b;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            a[e] = pack_bf16x2(large(half_of(a[e]), sign), large(half_of(a[e] >> 16), sign));
                            b[e] = pack_bf16x2(seen >> (8 * ks + 2 * e) & 1u ? BIG : 0.f,
                                               seen >> (8 * ks + 2 * e + 1) & 1u ? BIG : 0.f);
                        }
                        mma32<bf16_t>(z, a, b);
                    }
                    acc[dt] += z;
                }
        }
    }
    __device__ __forceinline__ static float half_of(uint32_t x) {
        if constexpr (std::is_same_v<T, bf16_t>) return __uint_as_float(x << 16);
        else return (float)__builtin_bit_cast(_Float16, (uint16_t)x);
    }
};

// Asks for an order of the block's instructions: the LDS reads of AHEAD products
// (READS each) before the first of N products, then with each product the reads of
// the one that far behind it.
template <int READS, int N, int AHEAD>
__device__ __forceinline__ void reads_ahead() {
    constexpr int DS_READ = 0x100, MFMA = 0x8, FIRST = AHEAD < N ? AHEAD : N;
    __builtin_amdgcn_sched_group_barrier(DS_READ, READS * FIRST, 0);
#pragma unroll
    for (int i = 0; i < N - FIRST; ++i) {
        __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
        __builtin_amdgcn_sched_group_barrier(DS_READ, READS, 0);
    }
    __builtin_amdgcn_sched_group_barrier(MFMA, FIRST, 0);
}

// ---- staging ---------------------------------------------------------------------

// Copies of PIECES KiB per wave, global -> LDS: lane l's 16 bytes at base + off[i]
// land at lds + i * step + 16 l.  Offsets at or past `bytes` touch no memory.
// Inline assembly, so that the compiler does not make later LDS reads wait for it:
// completion is awaited by the caller (vmcnt, then a barrier).  M0 holds the LDS
// address and is put back.
template <int PIECES, int STEP>
__device__ __forceinline__ void stage(const char *base, uint32_t bytes, const uint32_t (&off)[PIECES], uint32_t lds) {
    u32x4_t rsrc;
    const uint64_t b = (uint64_t)(uintptr_t)base;
    rsrc[0] = __builtin_amdgcn_readfirstlane((uint32_t)b);
    rsrc[1] = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xFFFFu);
    rsrc[2] = __builtin_amdgcn_readfirstlane(bytes);
    rsrc[3] = 0x00020000u;
    lds = __builtin_amdgcn_readfirstlane(lds);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        uint32_t saved;
        asm volatile(
            "s_mov_b32 %0, m0\n\t"
            "s_mov_b32 m0, %3\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %1, %2, 0 offen lds\n\t"
            "s_nop 0\n\t"
            "s_mov_b32 m0, %0"
            : "=&s"(saved)
            : "v"(off[i]), "s"(rsrc), "s"(lds + i * STEP)
            : "memory");
    }
}
__device__ __forceinline__ void staged_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Waits for the loads that fill x here.  Otherwise the wait would stand in the loop
// that uses it first, and there it would wait for the staging copies as well.
__device__ __forceinline__ void arrived(u32x4_t &x) { asm volatile("" : "+v"(x)); }
__device__ __forceinline__ void arrived(float &x) { asm volatile("" : "+v"(x)); }

// Whether a lane's sums are not all finite: 0 times a hidden infinity or NaN is NaN,
// so where they are, nothing of the kind has come in.
template <int N>
__device__ __forceinline__ bool any_not_finite(const f32x16_t (&acc)[N]) {
    bool bad = false;
#pragma unroll
    for (int dt = 0; dt < N; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) bad |= !(fabsf(acc[dt][i]) < __builtin_inff());
    return bad;
}

// The two halves' values of a lane's column joined.
__device__ __forceinline__ float half_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A lane's column of a transposed D x 32 result, times f, to a row of D elements.
// Elements 4 a .. 4 a + 3 of tile dt are columns 32 dt + 8 a + 4 h .. +3: the halves
// exchange, so that each stores 16 bytes.
template <typename T, int D>
__device__ __forceinline__ void store_column(T *row, const f32x16_t (&acc)[D / 32], float f, bool on) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) {
        if constexpr (std::is_same_v<T, float>) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                float4_t x;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = acc[dt][4 * a + e] * f;
                if (on) *reinterpret_cast<float4_t *>(row + 32 * dt + 8 * a + 4 * h) = x;
            }
        } else {
#pragma unroll
            for (int a = 0; a < 4; a += 2) {
                uint32_t x[2][2];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        x[b][e] = pack2<T>(acc[dt][4 * (a + b) + 2 * e] * f, acc[dt][4 * (a + b) + 2 * e + 1] * f);
                const auto p = __builtin_amdgcn_permlane32_swap(x[0][0], x[1][0], false, false);
                const auto q = __builtin_amdgcn_permlane32_swap(x[0][1], x[1][1], false, false);
                if (on) *reinterpret_cast<u32x4_t *>(row + 32 * dt + 8 * a + 8 * h) = u32x4_t{p[0], q[0], p[1], q[1]};
            }
        }
    }
}

// Lets a kernel have `bytes` of dynamic LDS.
template <typename K>
hipError_t swa_lds(K *kernel, int bytes) {
    if (bytes <= 65536) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// f(T{}, integral_constant<D>{}) for the call's element type and head dim.
template <bool D256, typename F>
hipError_t swa_with(int32_t dtype, int32_t dim, F f) {
    auto with_dim = [&](auto t) {
        using T = decltype(t);
        switch (dim) {
            case 32: return f(t, std::integral_constant<int, 32>{});
            case 64: return f(t, std::integral_constant<int, 64>{});
            case 128: return f(t, std::integral_constant<int, 128>{});
        }
        if constexpr (D256 && !std::is_same_v<T, float>)
            if (dim == 256) return f(t, std::integral_constant<int, 256>{});
        return hipErrorInvalidValue;
    };
    if (dtype == DT_BF16) return with_dim(bf16_t{});
    if (dtype == DT_FP16) return with_dim(_Float16{});
    return with_dim(float{});
}

}  // namespace gdn
