// Moves of resident states between slots, in place:
//   new[l, dst[m]] = old[l, src[m]], zeros where src[m] = -1
// with every source read before any destination is written, so sources and
// destinations may be the same slots in any pattern.
//
// A block owns a column tile: the same few bytes of every page of a layer.
// Moves never mix columns, so no block reads what another writes, and inside
// a block a barrier between its last load and its first store is all the
// ordering that chains and cycles need.  The tile is as wide as the block's
// registers allow: threads * kMoveVec vectors over all moves.
//
// Every block checks src and dst itself (they are a few KiB, in L2), so a bad
// index makes all of them write nothing without a second launch.
#include "gdn_ops.h"
#include "gdn_device.h"

namespace gdn {

constexpr int kMoveVec = 16;   // vectors a thread holds

template <typename vec_t, int NT>
__global__ __launch_bounds__(NT) void state_move_kernel(int slots, int moves, int64_t page_vecs, int lg_width,
                                                        vec_t *__restrict__ state, const int32_t *__restrict__ src,
                                                        const int32_t *__restrict__ dst, int32_t *__restrict__ status,
                                                        int layers) {
    __shared__ uint32_t seen[kMoveMaxSlots / 32];
    __shared__ int s_code;
    const int tid = threadIdx.x;
    for (int i = tid; i < (slots + 31) / 32; i += NT) seen[i] = 0u;
    if (tid == 0) s_code = 0;
    __syncthreads();
    int code = 0;
    for (int m = tid; m < moves; m += NT) {
        const int a = src[m], b = dst[m];
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

    const int width = 1 << lg_width, total = moves << lg_width;   // total <= NT * kMoveVec
    const int64_t col0 = (int64_t)blockIdx.x << lg_width;
    vec_t *base = state + (int64_t)blockIdx.y * slots * page_vecs;
    vec_t held[kMoveVec];
#pragma unroll
    for (int r = 0; r < kMoveVec; ++r) {
        const int i = tid + r * NT;
        const int64_t col = col0 + (i & (width - 1));
        held[r] = vec_t{};
        if (i < total && col < page_vecs) {
            const int a = src[i >> lg_width];
            if (a >= 0) held[r] = base[a * page_vecs + col];
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kMoveVec; ++r) {
        const int i = tid + r * NT;
        const int64_t col = col0 + (i & (width - 1));
        if (i < total && col < page_vecs) base[dst[i >> lg_width] * page_vecs + col] = held[r];
    }
}

hipError_t launch_state_move(const MoveArgs &a, hipStream_t st) {
    if ((a.moves == 0 || a.layers == 0) && !a.status) return hipSuccess;
    ProfScope prof("gdn_state_move", st);
    const bool wide = a.page_bytes % 16 == 0;
    const int64_t vecs = a.page_bytes / (wide ? 16 : 4);
    const int nt = a.moves <= 1024 ? 256 : 1024;
    int lg = 0;
    while (lg < 12 && ((int64_t)(a.moves ? a.moves : 1) << (lg + 1)) <= (int64_t)nt * kMoveVec &&
           ((int64_t)1 << lg) < vecs)
        ++lg;
    const int64_t tiles = (vecs + ((int64_t)1 << lg) - 1) >> lg;
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    for (int l0 = 0; l0 == 0 || l0 < a.layers; l0 += 65535) {
        const int nl = a.layers - l0 < 65535 ? a.layers - l0 : 65535;
        const dim3 grid((unsigned)(a.layers && a.moves ? tiles : 1), (unsigned)(nl > 0 ? nl : 1));
        auto go = [&](auto v, auto n) {
            using vec_t = decltype(v);
            state_move_kernel<vec_t, decltype(n)::value><<<grid, decltype(n)::value, 0, st>>>(
                a.slots, a.moves, vecs, lg, static_cast<vec_t *>(a.state) + (int64_t)l0 * a.slots * vecs, a.src,
                a.dst, a.status, a.layers);
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
