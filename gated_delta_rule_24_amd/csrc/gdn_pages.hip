// Moves of resident states between slots, in place:
//   new[l, dst[m]] = old[l, src[m]], zeros where src[m] = -1
// with every source read before any destination is written, so sources and
// destinations may be the same slots in any pattern.
//
// Every block checks src and dst itself (they are a few KiB, in L2), so a bad
// index makes all of them write nothing without a second launch; and it learns
// whether any destination is another move's source.
//   None is: the moves are one long copy, shared out in contiguous pieces.
//   Some are: a block owns a column tile, the same few bytes of every page of
// a layer.  Moves never mix columns, so no block reads what another writes, and
// inside a block a barrier between its last load and its first store is all the
// ordering that chains and cycles need.  The tile is as wide as the block's
// registers allow: NT * kMoveVec vectors over all moves.
// 96 pages of 1 MiB in 4 layers (0.81 GB read and written): pieces 149 us (5.4
// TB/s, the rate of a large copy), column tiles 159 us.
#include "gdn_device.h"
#include "gdn_ops.h"

#include <algorithm>

namespace gdn {

constexpr int kMoveVec = 16;   // vectors a thread holds of a column tile
constexpr int kMovePiece = 4;  // and of a piece

template <typename vec_t, int NT>
__global__ __launch_bounds__(NT) void state_move_kernel(int layers, int slots, int moves, int64_t page_vecs,
                                                        int lg_width, vec_t *__restrict__ state,
                                                        const int32_t *__restrict__ src,
                                                        const int32_t *__restrict__ dst,
                                                        int32_t *__restrict__ status) {
    extern __shared__ int s_idx[];             // src, dst, a bit per slot
    __shared__ int s_code, s_both;
    int *s_src = s_idx, *s_dst = s_idx + moves;
    uint32_t *seen = reinterpret_cast<uint32_t *>(s_idx + 2 * moves);
    const int tid = threadIdx.x;
    for (int i = tid; i < (slots + 31) / 32; i += NT) seen[i] = 0u;
    if (tid == 0) s_code = s_both = 0;
    __syncthreads();
    int code = 0;
    for (int m = tid; m < moves; m += NT) {
        const int a = src[m], b = dst[m];
        s_src[m] = a;
        s_dst[m] = b;
        if (a < -1 || a >= slots) code |= 1;
        if (b < 0 || b >= slots)
            code |= 2;
        else if (atomicOr(&seen[b >> 5], 1u << (b & 31)) & (1u << (b & 31)))
            code |= 4;
    }
    if (code) atomicOr(&s_code, code);
    __syncthreads();
    code = s_code;
    if (status && blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) {
        status[0] = moves;
        status[1] = (code & 1) ? 1 : ((code & 2) ? 2 : ((code & 4) ? 3 : 0));
    }
    if (code || layers == 0) return;
    for (int m = tid; m < moves; m += NT) {
        const int a = s_src[m];
        if (a >= 0 && a != s_dst[m] && (seen[a >> 5] >> (a & 31) & 1u)) s_both = 1;
    }
    __syncthreads();
    const bool both = s_both;
    vec_t *base = state + (int64_t)blockIdx.y * slots * page_vecs;

    if (!both) {
        constexpr int U = kMovePiece;
        for (int64_t p = (int64_t)blockIdx.x * NT * U; p < moves * page_vecs; p += (int64_t)gridDim.x * NT * U) {
            const int m0 = (int)(p / page_vecs);
            const int64_t c0 = p - m0 * page_vecs;
            vec_t v[U];
            int64_t to[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // loads without a branch, so that all are in flight together
                int64_t c = c0 + u * NT + tid;
                int m = m0;
                if (page_vecs >= NT * U) {
                    if (c >= page_vecs) c -= page_vecs, ++m;
                } else {
                    const uint32_t q = (uint32_t)c / (uint32_t)page_vecs;
                    c -= q * page_vecs;
                    m += q;
                }
                const int a = m < moves ? s_src[m] : -1, b = m < moves ? s_dst[m] : -1;
                v[u] = base[a >= 0 ? a * page_vecs + c : 0];
                if (a < 0) v[u] = vec_t{};
                to[u] = b >= 0 && a != b ? b * page_vecs + c : -1;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (to[u] >= 0) __builtin_nontemporal_store(v[u], base + to[u]);
        }
        return;
    }

    const int width = 1 << lg_width, total = moves << lg_width;   // total <= NT * kMoveVec
    for (int64_t tile = blockIdx.x; tile << lg_width < page_vecs; tile += gridDim.x) {
        const int64_t c0 = tile << lg_width;
        auto place = [&](int i, int &m, int64_t &c) {
            m = i >> lg_width;
            c = c0 + (i & (width - 1));
            return i < total && c < page_vecs;
        };
        vec_t held[kMoveVec];
        int t = tid;
#pragma unroll
        for (int r = 0; r < kMoveVec; ++r) {
            int m;
            int64_t c;
            const bool in = place(t + r * NT, m, c);
            const int a = in ? s_src[m] : -1;
            held[r] = base[a >= 0 ? a * page_vecs + c : 0];
            if (a < 0) held[r] = vec_t{};
        }
        __syncthreads();
        asm volatile("" : "+v"(t));      // places are worked out again, not kept
#pragma unroll
        for (int r = 0; r < kMoveVec; ++r) {
            int m;
            int64_t c;
            if (place(t + r * NT, m, c)) base[s_dst[m] * page_vecs + c] = held[r];
        }
    }
}

hipError_t launch_state_move(const MoveArgs &a, hipStream_t st) {
    if ((a.moves == 0 || a.layers == 0) && !a.status) return hipSuccess;
    ProfScope prof("gdn_state_move", st);
    const bool wide = a.page_bytes % 16 == 0;
    const int64_t vecs = a.page_bytes / (wide ? 16 : 4);
    // Wide blocks where the moves are many, so that a column tile stays at
    // least 64 bytes wide; 16 bytes where pages are no whole 16-byte vectors.
    // Measured, a rotation of 2000 and 4000 pages: 16384 bytes long 16 and 53
    // us, 16388 bytes 55 and 185 (a copy 12 and 24).  A rotation of few pages
    // has few tiles, 32 for two pages of 1 MiB; with 2 to 16 pages it takes 6.5
    // to 7.5 us, of which the call is about 6.
    const int nt = a.moves <= 1024 ? 256 : 1024;
    const size_t lds = 4 * (2 * (size_t)a.moves + (a.slots + 31) / 32);
    int lg = 0;
    while (((int64_t)std::max(a.moves, 1) << (lg + 1)) <= (int64_t)nt * kMoveVec && ((int64_t)1 << lg) < vecs) ++lg;
    // A block looks through all indices before it moves anything, so it takes
    // two pieces where that leaves enough blocks for all CUs, and more above
    // 16384 blocks.  Measured, 64 forks of 1 MiB (4096 pieces): 2048 blocks
    // 16.8 us, 4096 19.1; 96 pages in 4 layers (24576 pieces): 2048 blocks 160
    // us, 12288 155, 16384 148, 24576 148.
    const int64_t layers = std::max(a.layers, 1);
    const int64_t pieces = (a.moves * vecs + nt * kMovePiece - 1) / (nt * kMovePiece), all = pieces * layers;
    const int64_t blocks = all > 8192 ? std::max<int64_t>(std::min(pieces, 16384 / layers), 16)
                           : all > 1024 ? (pieces + 1) / 2
                                        : pieces;
    for (int l0 = 0; l0 == 0 || l0 < a.layers; l0 += 65535) {
        const int nl = std::max(std::min(a.layers - l0, 65535), 1);
        const dim3 grid((unsigned)std::max<int64_t>(a.layers ? blocks : 1, 1), (unsigned)nl);
        auto go = [&](auto v, auto n) {
            using vec_t = decltype(v);
            state_move_kernel<vec_t, decltype(n)::value><<<grid, decltype(n)::value, lds, st>>>(
                a.layers, a.slots, a.moves, vecs, lg,
                static_cast<vec_t *>(a.state) + (int64_t)l0 * a.slots * vecs, a.src, a.dst, a.status);
        };
        using std::integral_constant;
        if (wide) {
            if (nt == 256) go(float4_t{}, integral_constant<int, 256>{});
            else go(float4_t{}, integral_constant<int, 1024>{});
        } else {
            if (nt == 256) go(float{}, integral_constant<int, 256>{});
            else go(float{}, integral_constant<int, 1024>{});
        }
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace gdn
