// Internal interface between the C ABI (gdn_ops_api.cpp) and the kernels of
// the gated linear recurrence, layer norm and the state moves.  Arguments
// arrive here already validated.
#pragma once

#include "gdn_launch.h"

#include <type_traits>

namespace gdn {

// Types of one call: each fp32 or one 16-bit type.
struct ScanArgs {
    int32_t B, T, D, N, in_dtype, gate_dtype, out_dtype;
    const void *x, *log_alpha;     // forward
    const float *init_state;
    const int32_t *cu_seqlens;
    void *h;                       // forward: written; backward: read
    float *final_state;
    const void *d_h;               // backward
    const float *d_final;
    void *dx, *dlog_alpha;
    float *d_init;
    void *workspace;
};

// Workspace carve-up of one scan call (byte offsets).
struct ScanWorkspace {
    int64_t rows, chunks, tiles;   // chains = rows * tiles of channels, chunks = tiles of tokens per chain
    size_t off_seq, off_init, off_agg, off_grp, off_pre;
    size_t total;
};
ScanWorkspace scan_workspace_layout(int32_t B, int32_t T, int32_t D, int32_t N, bool packed);

struct ScanStepArgs {
    int32_t N, D, in_dtype, gate_dtype, out_dtype;
    float *state;
    const void *x, *log_alpha;
    void *h;
};

hipError_t launch_scan_fwd(const ScanArgs &a, hipStream_t stream);
hipError_t launch_scan_bwd(const ScanArgs &a, hipStream_t stream);
hipError_t launch_scan_step(const ScanStepArgs &a, hipStream_t stream);

constexpr int kNormMaxDim = 16384;
struct NormArgs {
    int64_t rows;
    int32_t dim, in_dtype, out_dtype;
    float eps;
    const void *x;
    const float *weight, *bias;
    void *y;                       // forward
    float *mean, *rstd;            // forward: written; backward: read
    const void *dy;                // backward
    void *dx;
    float *dweight, *dbias;
    void *workspace;
};
size_t layernorm_bwd_workspace(int64_t rows, int32_t dim);
hipError_t launch_layernorm_fwd(const NormArgs &a, hipStream_t stream);
hipError_t launch_layernorm_bwd(const NormArgs &a, hipStream_t stream);

constexpr int kMoveMaxSlots = 65536, kMoveMaxMoves = 4096;
struct MoveArgs {
    int32_t layers, slots, moves;
    int64_t page_bytes;
    void *state;
    const int32_t *src, *dst;
    int32_t *status;
};
hipError_t launch_state_move(const MoveArgs &a, hipStream_t stream);


}  // namespace gdn
