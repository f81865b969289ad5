/*
 * gdn.h -- C ABI of the gated delta rule layer core for MI355X (gfx950).
 *
 * The operation (Gated Delta Networks paper, section 3.1, eq. (10)):
 *
 *     S_t = S_{t-1} ( alpha_t (I - beta_t k_t k_t^T) ) + beta_t v_t k_t^T
 *     o_t = S_t q_t                      S_t in R^{dv x dk},  alpha_t = exp(log_alpha_t)
 *
 * evaluated two ways:
 *   gdn_chunk_fwd    -- chunkwise-parallel prefill over whole sequences
 *                       (paper section 3.3, the WY/UT chunk algorithm with the
 *                       decay mask; paper-notes blog, "Hardware-Efficient
 *                       Chunkwise Training", summary (4)), optionally packed
 *                       with cu_seqlens, from an initial state, returning the
 *                       final state.
 *   gdn_decode_step  -- one token of the recurrence for a batch of resident
 *                       states, updated in place (tutorial page, decode
 *                       recursion S_t = S_{t-1} A_t + B_t).
 * and differentiated:
 *   gdn_chunk_bwd    -- gradients of gdn_chunk_fwd's outputs with respect to
 *                       all of its inputs (for training).
 * gdn_chunk_fwd_noalloc is gdn_chunk_fwd for callers that cannot allocate
 * device memory: it uses a scratch array of the library instead of a
 * workspace argument.
 *
 * Next to it, in the same conventions: the elementwise gated linear
 * recurrence (gdn_scan_fwd, gdn_scan_bwd, gdn_scan_step), layer norm
 * (gdn_layernorm_fwd, gdn_layernorm_bwd) and moves of resident states
 * (gdn_state_move), described at their declarations.
 *
 * Both evaluations return the same numbers as the recurrence up to floating-point
 * rounding.  Chunked, single-step and save-then-resume evaluations agree
 * (tutorial: the three paths must line up; independent samples reset the
 * state, a continued request does not).
 *
 * CONVENTIONS (all calls)
 *   - Every pointer argument except `stream` is a DEVICE pointer (HBM) unless
 *     stated otherwise.  Tensors are dense, row-major, last index fastest.
 *   - The caller owns every buffer.  The library keeps no pointer after the
 *     call returns and allocates no device memory on these paths (the one
 *     device array it owns is gdn_chunk_fwd_noalloc's scratch array, which
 *     exists while the library is loaded).
 *   - Work is enqueued on `stream` (NULL = the default stream) and the call
 *     returns without waiting.  Buffers must stay valid until the stream
 *     reaches that point.  A kernel fault shows up at the caller's next
 *     synchronisation, as for any HIP launch.
 *   - All argument checks run before anything is enqueued: a call that
 *     returns an error status has launched nothing and written nothing.
 *     gdn_last_error_message() then describes the failure (thread-local).
 *   - q, k, v, o, the state buffers and the workspace must be 16-byte
 *     aligned; log_alpha, beta and cu_seqlens 4-byte aligned
 *     (GDN_ERR_ALIGN otherwise).
 *   - Calls are reentrant and may run concurrently on different streams with
 *     disjoint buffers.
 *   - Preconditions that are documented but NOT checked on the device:
 *     finite inputs; log_alpha <= 0; beta in [0, 1] (any finite beta is
 *     computed as given); q and k normalised upstream (the paper normalises
 *     them in the token-mixing block, section 3.4).  With 16-bit inputs the
 *     matrix-core operands are fp16, so |q|, |k|, |v| and the state entries
 *     must stay below 65504.  Outside that range nothing reports an error:
 *     bf16 q, k and v reach their fp16 operands through a round-toward-zero
 *     conversion and saturate silently at +-65504, and a state entry that is
 *     rounded to an fp16 operand (round to nearest) becomes infinite.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 5

typedef enum {
    GDN_OK = 0,
    GDN_ERR_NULL = 1,         /* a required pointer is NULL                       */
    GDN_ERR_SHAPE = 2,        /* sizes negative, zero where not allowed, or
                                 inconsistent                                     */
    GDN_ERR_DTYPE = 3,        /* unknown dtype code                               */
    GDN_ERR_ALIGN = 4,        /* a device pointer is misaligned (see CONVENTIONS) */
    GDN_ERR_UNSUPPORTED = 5,  /* well-formed but not built (head dims, chunk size,
                                 dtype combination)                               */
    GDN_ERR_WORKSPACE = 6,    /* workspace NULL or smaller than required          */
    GDN_ERR_HIP = 7,          /* a HIP runtime call or launch failed              */
    GDN_ERR_ALIAS = 8,        /* an output overlaps an input it may not overlap   */
    GDN_ERR_DEVICE_INPUT = 9  /* device-side validation failed (gdn_chunk_fwd_check) */
} gdn_status;

typedef enum {
    GDN_FP32 = 0,
    GDN_BF16 = 1,
    GDN_FP16 = 2
} gdn_dtype;

/*
 * Options of gdn_chunk_fwd (gdn_chunk_desc.flags) and gdn_decode_step.
 *   GDN_QK_L2NORM  q and k are L2-normalised per (token, head) inside the
 *                  kernels, q / ||q||_2 and k / ||k||_2, as the Gated
 *                  DeltaNet paper's token-mixing block does before the delta
 *                  rule (section 3.4, "Token mixer block"; the paper notes
 *                  list it for training stability).  The input buffers are
 *                  not modified.  An all-zero vector stays zero.
 */
typedef enum {
    GDN_QK_L2NORM = 1
} gdn_flags;

/*
 * Shape of one gdn_chunk_fwd call.
 *   batch     B  >= 1: batch rows.  Must be 1 when cu_seqlens is given.
 *   seqlen    T  >= 0: tokens per batch row (packed batch: total tokens).
 *   heads     H  >= 1.
 *   dk           key/query head dim: 32, 64, 128 or 256 (fp32 inputs: <= 128).
 *   dv           value head dim: a multiple of 16, 16..1024.
 *   num_seqs  N: number of sequences.  Without cu_seqlens it must equal B
 *                (row b is sequence b); with cu_seqlens, N >= 1 and the
 *                cu_seqlens array holds N+1 offsets.
 *   chunk     C: chunk length; 64 is the supported value.
 *   in_dtype     dtype of q, k, v (FP32, BF16 or FP16).  BF16/FP16 inputs run
 *                the matrix products on fp16 operands with fp32 accumulation
 *                and an fp32 state; FP32 inputs run them on fp32 operands.
 *   out_dtype    dtype of o (FP32, BF16 or FP16).
 *   flags        bitwise OR of gdn_flags (0: none).
 */
typedef struct {
    int32_t batch;
    int32_t seqlen;
    int32_t heads;
    int32_t dk;
    int32_t dv;
    int32_t num_seqs;
    int32_t chunk;
    int32_t in_dtype;   /* gdn_dtype */
    int32_t out_dtype;  /* gdn_dtype */
    int32_t flags;      /* gdn_flags */
} gdn_chunk_desc;

/* ABI version of the loaded library (GDN_ABI_VERSION at build time). */
int gdn_abi_version(void);

/* Static, human-readable name of a status code. */
const char *gdn_status_string(gdn_status status);

/* Detail of the last failed call on this thread ("" if none).  The pointer is
 * valid until the next gdn_* call on the same thread. */
const char *gdn_last_error_message(void);

/*
 * Workspace for gdn_chunk_fwd, in bytes, written to *bytes (host pointer).
 * Depends only on the descriptor (and on GDN_SEG_CHUNKS, below).  The
 * workspace holds the chunk table built from cu_seqlens and, per (chunk,
 * head), the UT-transform matrix T diag(beta), the decay-masked Q K^T block
 * and the chunk's decay factors (exp of the cumulative log-decay from the
 * chunk start, and to the chunk end).  When the state pass is segmented (a
 * batch with too few (sequence, head) pairs to fill the GPU: each sequence's
 * chunks are cut into segments whose affine state maps S -> S F + G are
 * formed in parallel and then chained, the algebra of the paper's chunk-level
 * state recurrence, section 3.3, applied to runs of chunks) it also holds the
 * segment table and, per (segment, head), the map [G; F] ((dv + dk) x dk
 * fp32) and the segment's incoming state (dv x dk fp32).  The environment
 * variable GDN_SEG_CHUNKS, read at every call, fixes the segment length in
 * chunks (0 = never segment); unset, the library chooses.  The workspace
 * need not be initialised and may be reused by later calls that are ordered
 * after this one on the stream.
 * Errors: GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_UNSUPPORTED.
 */
gdn_status gdn_chunk_fwd_workspace_size(const gdn_chunk_desc *desc, size_t *bytes);

/*
 * Chunkwise-parallel forward pass (prefill).
 *
 *   q           [B, T, H, dk]  in_dtype
 *   k           [B, T, H, dk]  in_dtype
 *   v           [B, T, H, dv]  in_dtype
 *   log_alpha   [B, T, H]      fp32, log of the forget gate alpha_t
 *   beta        [B, T, H]      fp32, write strength beta_t
 *   init_state  [N, H, dv, dk] fp32 or NULL (zeros).  S[n,h] maps keys to
 *                              values, row index = value dim (paper 2.1).
 *   cu_seqlens  int32 [N+1] or NULL.  Packed batch (B == 1): sequence n is
 *               tokens cu[n] .. cu[n+1]-1 of the T axis; cu[0] = 0,
 *               non-decreasing, cu[N] = T.  Empty sequences are allowed
 *               (their final state equals their initial state).  The state
 *               restarts from init_state[n] at every sequence start, and
 *               chunks restart there too (the last chunk of a sequence may
 *               be partial).  The array is checked on the device; a
 *               malformed one makes the kernels write nothing and is
 *               reported by gdn_chunk_fwd_check.
 *   o           [B, T, H, dv]  out_dtype (written)
 *   final_state [N, H, dv, dk] fp32 or NULL (not returned).  May be the
 *               same pointer as init_state (in-place continuation): each
 *               state tile is read before it is written and tiles are
 *               disjoint.  Partial overlap with init_state is not allowed.
 *   workspace   device buffer of at least gdn_chunk_fwd_workspace_size bytes
 *   stream      HIP stream the kernels are launched on
 *
 * Evaluation: when the call averages more than 16 tokens per sequence
 * (B*T > 16*N) it runs the chunkwise algorithm (paper section 3.3) with
 * 64-token chunks.  Otherwise each (sequence, head) state is read and
 * written once by one kernel: for 16-bit inputs with dk <= 128 the same
 * chunkwise algorithm with 16-token chunks on the matrix cores, else the
 * recurrence itself token by token; either is cheaper for a few tokens per
 * sequence.  The environment variable GDN_SMALL_CHUNKS=0, read at every
 * call, sends such calls to the token-by-token kernel.  All compute eq. (10)
 * with fp32 state and accumulation and meet the same bounds; bit-identical
 * results are guaranteed between calls that take the same branch.
 *
 * o must not overlap any input or the state buffers (GDN_ERR_ALIAS).
 * Errors: GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_ALIGN,
 * GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE, GDN_ERR_ALIAS, GDN_ERR_HIP.
 */
gdn_status gdn_chunk_fwd(const gdn_chunk_desc *desc,
                         const void *q, const void *k, const void *v,
                         const float *log_alpha, const float *beta,
                         const float *init_state, const int32_t *cu_seqlens,
                         void *o, float *final_state,
                         void *workspace, size_t workspace_bytes,
                         hipStream_t stream);

/*
 * gdn_chunk_fwd for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc).
 * Same arguments, semantics and errors as gdn_chunk_fwd, without the
 * workspace: the library's own scratch array stands in for it, a
 * GDN_NOALLOC_SCRATCH_BYTES device array per GPU that exists from the moment
 * the library is loaded until the process ends.  Its device address is
 * looked up (hipGetSymbolAddress) on the first call on each device; the call
 * itself allocates nothing.
 *   - A call whose gdn_chunk_fwd_workspace_size exceeds
 *     GDN_NOALLOC_SCRATCH_BYTES returns GDN_ERR_WORKSPACE and writes nothing
 *     (64 MiB covers, e.g., B = 4, T = 4096, H = 16, dk = dv = 128 with
 *     16-bit inputs).
 *   - Every call on a GPU uses that GPU's one array.  Calls that may overlap
 *     in time on one GPU (different streams, or different host threads
 *     without ordering) race on it and must not be issued; calls ordered on
 *     one stream are safe.  Nothing in the array has to start at a known
 *     value: each call writes every part of it that it reads.
 *   - A malformed cu_seqlens makes the kernels write nothing, as in
 *     gdn_chunk_fwd, but is not reported (gdn_chunk_fwd_check needs the
 *     workspace pointer).
 */
#define GDN_NOALLOC_SCRATCH_BYTES (64u << 20)
gdn_status gdn_chunk_fwd_noalloc(const gdn_chunk_desc *desc,
                                 const void *q, const void *k, const void *v,
                                 const float *log_alpha, const float *beta,
                                 const float *init_state, const int32_t *cu_seqlens,
                                 void *o, float *final_state, hipStream_t stream);

/*
 * Workspace for gdn_chunk_bwd, in bytes, written to *bytes (host pointer).
 * Depends only on the descriptor.  Besides the chunk table it holds, per
 * (chunk, head), the fp32 UT-transform matrix T = (I + A)^{-1}, the
 * decay-masked Q K^T and K K^T blocks and the decay vectors (49 KiB at
 * C = 64), the
 * state and the state's gradient at every chunk boundary (2 * dv * dk * 4
 * bytes) and three C x dv fp32 chunk intermediates.  Prefill with B = 4,
 * T = 4096, H = 16, dk = dv = 128 needs about 1 GiB.  With GDN_QK_L2NORM
 * in desc->flags it also holds the normalised q and k and v as fp32 rows and
 * the two normalisation factors, (2 dk + dv + 2) * 4 bytes per (token, head).
 * Errors: GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_UNSUPPORTED.
 */
gdn_status gdn_chunk_bwd_workspace_size(const gdn_chunk_desc *desc, size_t *bytes);

/*
 * Backward pass of gdn_chunk_fwd: given the gradients of a loss with respect
 * to o and to the final state, the gradients with respect to every input.
 * The pages call the chunkwise algorithm a training method (paper section
 * 3.3) but give no gradient formulas; these follow from differentiating the
 * recurrence of eq. (10), evaluated on the chunked form.  The forward pass
 * is recomputed from the inputs (nothing from gdn_chunk_fwd is kept).
 *
 *   desc, q, k, v, log_alpha, beta, init_state, cu_seqlens
 *               as for gdn_chunk_fwd (desc->out_dtype is not used)
 *   d_o            [B, T, H, dv]  fp32, dL/do
 *   d_final_state  [N, H, dv, dk] fp32 or NULL (zeros): dL/d final state
 *   dq, dk         [B, T, H, dk]  fp32 (written)
 *   dv             [B, T, H, dv]  fp32 (written)
 *   dlog_alpha     [B, T, H]      fp32 (written), dL/d log_alpha
 *   dbeta          [B, T, H]      fp32 (written)
 *   d_init_state   [N, H, dv, dk] fp32 or NULL (not returned): dL/d init_state
 *                  (with init_state NULL it is the gradient at a zero state)
 *   workspace      at least gdn_chunk_bwd_workspace_size bytes
 *
 * Supported: dk 32, 64 or 128; dv a multiple of 16 up to 1024; flags 0 or
 * GDN_QK_L2NORM.  With GDN_QK_L2NORM the gradients are those of the call
 * that normalised q and k (paper section 3.4, token mixer block): the
 * backward kernels run on q^ = q / ||q||, k^ = k / ||k|| (fp32 rows in the
 * workspace) and dq, dk are carried back through the normalisation,
 * dx = (dx^ - x^ (x^ . dx^)) / ||x||, zero for an all-zero row.  All
 * gradient arithmetic has fp32 precision for every input dtype (products
 * with a 16-bit q or k factor may run on the 16-bit matrix cores with the
 * other factor split exactly into three bf16 terms).  Tokens past a
 * sequence's end are not written.  With cu_seqlens the array is checked on
 * the device as in gdn_chunk_fwd; a malformed one makes the kernels write
 * nothing and gdn_chunk_fwd_check(workspace, ...) reports it.
 * The outputs must not overlap each other, any input or the workspace
 * (GDN_ERR_ALIAS).
 * Errors: GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_ALIGN,
 * GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE, GDN_ERR_ALIAS, GDN_ERR_HIP.
 */
gdn_status gdn_chunk_bwd(const gdn_chunk_desc *desc,
                         const void *q, const void *k, const void *v,
                         const float *log_alpha, const float *beta,
                         const float *init_state, const int32_t *cu_seqlens,
                         const float *d_o, const float *d_final_state,
                         float *dq, float *dk, float *dv,
                         float *dlog_alpha, float *dbeta, float *d_init_state,
                         void *workspace, size_t workspace_bytes,
                         hipStream_t stream);

/*
 * Result of the device-side check of the last gdn_chunk_fwd (or packed
 * gdn_chunk_bwd, gdn_scan_fwd, gdn_scan_bwd) that used `workspace`, or of
 * the gdn_state_move that wrote it as its status (codes there).  Synchronises `stream`, then writes 0 (valid) or a
 * non-zero code (1: cu[0] != 0, 2: decreasing offsets, 3: cu[N] != T) to
 * *code (host pointer).  Returns GDN_ERR_DEVICE_INPUT when the code is
 * non-zero, GDN_OK otherwise.
 */
gdn_status gdn_chunk_fwd_check(const void *workspace, hipStream_t stream, int32_t *code);

/*
 * One decode step for N resident states, in place.
 *
 *   state      [N, H, dv, dk] fp32, read and overwritten with S_t
 *   q, k       [N, H, dk]     in_dtype
 *   v          [N, H, dv]     in_dtype
 *   log_alpha  [N, H]         fp32
 *   beta       [N, H]         fp32
 *   o          [N, H, dv]     out_dtype, o = S_t q (read after the update)
 *
 * Per (n, h) it computes, reading each state row once and writing it once:
 *   Sbar = alpha S;  u = beta (v - Sbar k);  S_t = Sbar + u k^T;
 *   o = alpha (S q) + u (k . q)
 * (tutorial page: forget first, then correct the error of the decayed
 * memory).  flags: 0 or GDN_QK_L2NORM (q and k normalised first).
 * dk: 32, 64, 128 or 256.  dv: 1..4096.
 * o must not overlap state.
 * Errors: GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_ALIGN,
 * GDN_ERR_UNSUPPORTED, GDN_ERR_ALIAS, GDN_ERR_HIP.
 */
gdn_status gdn_decode_step(int32_t N, int32_t H, int32_t dk, int32_t dv,
                           int32_t in_dtype, int32_t out_dtype, int32_t flags,
                           float *state,
                           const void *q, const void *k, const void *v,
                           const float *log_alpha, const float *beta,
                           void *o, hipStream_t stream);

/*
 * Gated linear recurrence: the elementwise sibling of the gated delta rule,
 * with a state of one value per channel,
 *
 *     h_t = alpha_t h_{t-1} + x_t          alpha_t = exp(log_alpha_t)
 *
 * over the tokens t of a sequence, each channel on its own.
 *   gdn_scan_fwd   -- whole sequences (prefill, training), optionally packed
 *                     with cu_seqlens, from an initial state, returning the
 *                     final state
 *   gdn_scan_bwd   -- gradients of gdn_scan_fwd's outputs
 *   gdn_scan_step  -- one token for a batch of resident states, in place
 *
 * Shape of a gdn_scan_fwd / gdn_scan_bwd call:
 *   batch       B >= 1: batch rows.  Must be 1 when cu_seqlens is given.
 *   seqlen      T >= 0: tokens per row (packed: total tokens); B * T < 2^30.
 *   channels    D: 1..65536 (a layer with heads passes heads * head dim).
 *   num_seqs    N: B without cu_seqlens; with it, cu_seqlens has N + 1
 *               offsets.
 *   in_dtype    dtype of x and of its gradient
 *   gate_dtype  dtype of log_alpha and of its gradient
 *   out_dtype   dtype of h and of its gradient
 *               Each is FP32 or one 16-bit type; BF16 and FP16 do not mix in
 *               one call (GDN_ERR_UNSUPPORTED).  States are fp32, and every
 *               state, decay and carry is held in fp32 whatever the types;
 *               an output is rounded once, to nearest, when it is stored.
 *   flags       0.
 */
typedef struct {
    int32_t batch;
    int32_t seqlen;
    int32_t channels;
    int32_t num_seqs;
    int32_t in_dtype;    /* gdn_dtype */
    int32_t gate_dtype;  /* gdn_dtype */
    int32_t out_dtype;   /* gdn_dtype */
    int32_t flags;
} gdn_scan_desc;

/*
 * Workspace for gdn_scan_fwd and gdn_scan_bwd, in bytes, written to *bytes
 * (host pointer).  Depends only on the descriptor.  Need not be initialised;
 * may be reused by later calls ordered after this one on the stream.
 * Errors: GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_UNSUPPORTED.
 */
gdn_status gdn_scan_workspace_size(const gdn_scan_desc *desc, size_t *bytes);

/*
 * Forward pass.
 *
 *   x            [B, T, D]  in_dtype
 *   log_alpha    [B, T, D]  gate_dtype, <= 0 (not checked; -inf forgets
 *                           everything.  Products of alpha over up to 8192
 *                           tokens are formed, and sums of what a tile adds
 *                           to a state of 0: with positive log_alpha, or x
 *                           next to the largest fp32 values, they may overflow
 *                           where the recurrence would not)
 *   init_state   [N, D]     fp32 or NULL (zeros)
 *   cu_seqlens   int32 [N+1] or NULL, as for gdn_chunk_fwd: empty sequences
 *                are allowed, a malformed array makes the kernels write
 *                nothing and gdn_chunk_fwd_check(workspace, ...) reports it
 *   h            [B, T, D]  out_dtype (written)
 *   final_state  [N, D]     fp32 or NULL (not returned).  May be the same
 *                           pointer as init_state (in-place continuation),
 *                           not a partial overlap.
 * Values that are not finite are carried as the recurrence carries them: an
 * infinite state stays infinite however long it decays, and becomes
 * not-a-number where alpha is 0 (log_alpha below -87.33 counts as that: alpha
 * has no values between 0 and 2^-126).
 * Nothing of one sequence reaches another, not-a-number and infinite values
 * included.  Equal calls give equal bits.  Long sequences are cut into tiles
 * whose blocks hand states on through the workspace; the environment variable
 * GDN_SCAN_PATIENCE, read at every call, sets how often a block looks for
 * another's word before it works the state out itself, with the same bits
 * (default 4096, about 4 ms; 0 makes every block do so where it can).
 * x, log_alpha, h, the states and the workspace must be 16-byte aligned.
 * h, final_state and the workspace must not overlap anything else
 * (GDN_ERR_ALIAS).
 * Errors: as gdn_chunk_fwd.
 */
gdn_status gdn_scan_fwd(const gdn_scan_desc *desc, const void *x, const void *log_alpha,
                        const float *init_state, const int32_t *cu_seqlens,
                        void *h, float *final_state,
                        void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Backward pass: gradients of a loss with respect to x, log_alpha and the
 * initial state, given those with respect to h and the final state.  With
 * g_t the whole gradient of h_t and e_t = alpha_t g_t,
 *     g_t = d_h_t + e_{t+1}     (d_h_L + d_final_state at a sequence's end)
 *     dx_t = g_t     dlog_alpha_t = e_t h_{t-1}     d_init_state = e_1
 *
 *   log_alpha, init_state, cu_seqlens   as for gdn_scan_fwd
 *   h              [B, T, D]  out_dtype, gdn_scan_fwd's output.  With a
 *                             16-bit out_dtype its rounding (half a step of
 *                             the type) carries over to dlog_alpha.
 *   d_h            [B, T, D]  out_dtype
 *   d_final_state  [N, D]     fp32 or NULL (zeros)
 *   dx             [B, T, D]  in_dtype (written)
 *   dlog_alpha     [B, T, D]  gate_dtype (written)
 *   d_init_state   [N, D]     fp32 or NULL (not returned); with init_state
 *                             NULL it is the gradient at a zero state.  Of an
 *                             empty sequence it is d_final_state.
 * The outputs must not overlap each other, any input or the workspace.
 * Errors: as gdn_chunk_bwd.
 */
gdn_status gdn_scan_bwd(const gdn_scan_desc *desc, const void *log_alpha, const void *h,
                        const float *init_state, const int32_t *cu_seqlens,
                        const void *d_h, const float *d_final_state,
                        void *dx, void *dlog_alpha, float *d_init_state,
                        void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One token for N resident states, in place.
 *
 *   state      [N, D]  fp32, read and overwritten with h_t
 *   x          [N, D]  in_dtype
 *   log_alpha  [N, D]  gate_dtype
 *   h          [N, D]  out_dtype (written), the new state rounded once
 * D: 1..65536; types as for gdn_scan_fwd.  N * D < 2^40.  h and state must
 * not overlap each other or an input.  N = 0 does nothing.
 * Errors: GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_ALIGN,
 * GDN_ERR_UNSUPPORTED, GDN_ERR_ALIAS, GDN_ERR_HIP.
 */
gdn_status gdn_scan_step(int32_t N, int32_t D, int32_t in_dtype, int32_t gate_dtype, int32_t out_dtype,
                         float *state, const void *x, const void *log_alpha, void *h, hipStream_t stream);

/*
 * Layer norm over the last dimension,
 *     mean = sum_i x_i / D     rstd = 1 / sqrt(sum_i (x_i - mean)^2 / D + eps)
 *     y_i = (x_i - mean) rstd weight_i + bias_i
 * as it stands behind the recurrence (per head, D = dv) or in front of the
 * block (D = model width).
 *
 *   rows       R >= 0, R < 2^31
 *   dim        D: 1..16384
 *   eps        finite and >= 0 (GDN_ERR_UNSUPPORTED otherwise)
 *   x          [R, D]  in_dtype
 *   weight     [D]     fp32 or NULL (ones)
 *   bias       [D]     fp32 or NULL (zeros)
 *   y          [R, D]  out_dtype (written)
 *   mean, rstd [R]     fp32 (written) or both NULL (not returned)
 * in_dtype and out_dtype: each FP32 or one 16-bit type, not BF16 with FP16.
 * Statistics are fp32 sums, the squares taken about the mean; y is rounded
 * once.  A row's results depend on that row alone.  With eps = 0 a constant
 * row has no finite rstd.
 * x, y, weight and bias must be 16-byte aligned, mean and rstd 4-byte.  The
 * outputs must not overlap each other or an input.
 * Errors: GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_ALIGN,
 * GDN_ERR_UNSUPPORTED, GDN_ERR_ALIAS, GDN_ERR_HIP.
 */
gdn_status gdn_layernorm_fwd(int64_t rows, int32_t dim, int32_t in_dtype, int32_t out_dtype, float eps,
                             const void *x, const float *weight, const float *bias,
                             void *y, float *mean, float *rstd, hipStream_t stream);

/*
 * Workspace of gdn_layernorm_bwd in bytes, written to *bytes (host pointer).
 * Need not be initialised.  Errors: GDN_ERR_NULL, GDN_ERR_SHAPE,
 * GDN_ERR_UNSUPPORTED.
 */
gdn_status gdn_layernorm_bwd_workspace_size(int64_t rows, int32_t dim, size_t *bytes);

/*
 * Gradients of gdn_layernorm_fwd.  With xh = (x - mean) rstd and
 * u = dy weight,
 *     dx = rstd (u - sum(u) / D - xh sum(u xh) / D)
 *     dweight = sum over rows of dy xh     dbias = sum over rows of dy
 *
 *   dy          [R, D]  out_dtype
 *   x           [R, D]  in_dtype
 *   mean, rstd  [R]     fp32, as gdn_layernorm_fwd gave them
 *   weight      [D]     fp32 or NULL (ones)
 *   dx          [R, D]  in_dtype (written)
 *   dweight     [D]     fp32 or NULL (not returned), written, not added to
 *   dbias       [D]     fp32 or NULL (not returned), written, not added to
 *   workspace   at least gdn_layernorm_bwd_workspace_size bytes, 16-byte
 *               aligned; may be NULL when neither dweight nor dbias is asked
 *               for
 * The sums over rows are taken in a fixed order: equal calls give equal
 * bits.  With R = 0 dweight and dbias are zeros.
 * The outputs must not overlap each other, any input or the workspace.
 * Errors: those of gdn_layernorm_fwd and GDN_ERR_WORKSPACE.
 */
gdn_status gdn_layernorm_bwd(int64_t rows, int32_t dim, int32_t in_dtype, int32_t out_dtype,
                             const void *dy, const void *x, const float *mean, const float *rstd,
                             const float *weight, void *dx, float *dweight, float *dbias,
                             void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Moves of resident states.  A page is the state of one sequence in one
 * layer: one slot of gdn_decode_step's or gdn_scan_step's state, page_bytes
 * long (fp32 [H, dv, dk]: 4 H dv dk).  For every layer l and every
 * m < moves,
 *     new[l, dst[m]] = old[l, src[m]]        zeros where src[m] = -1
 * with every source read as it was before the call, so that one call
 *   - forks a state (one source, many destinations),
 *   - compacts a batch after sequences have ended (live states into holes),
 *   - reorders or swaps states (cycles are fine),
 *   - frees slots for new sequences (src = -1).
 * Slots that are no destination keep their bytes.
 *
 *   layers      L >= 0
 *   slots       P: 1..65536
 *   page_bytes  a multiple of 4, >= 4
 *   moves       M: 0..min(P, 4096)
 *   state       [L, P, page_bytes], 16-byte aligned, updated in place
 *   src         int32 [M], each -1 or a slot
 *   dst         int32 [M], slots, no two alike
 *   status      int32 [2] or NULL (written): {M, code}.  src and dst are
 *               device data and are checked on the device: code 1 for a
 *               source out of range, 2 for a destination out of range, 3 for
 *               a destination given twice, 0 otherwise; where it is not 0
 *               the call changes nothing else.  gdn_chunk_fwd_check(status,
 *               ...) reads it.  src, dst, status: 4-byte aligned.
 * src, dst and status must not overlap the state or status an index array.
 * Errors: GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_ALIGN, GDN_ERR_UNSUPPORTED,
 * GDN_ERR_ALIAS, GDN_ERR_HIP.
 */
gdn_status gdn_state_move(int32_t layers, int32_t slots, int64_t page_bytes, int32_t moves,
                          void *state, const int32_t *src, const int32_t *dst, int32_t *status,
                          hipStream_t stream);

/*
 * Per-kernel timing for measurement harnesses (host-side bookkeeping only;
 * kernels are unchanged).  While enabled, every launch made by this library
 * is bracketed by a pair of HIP events recorded on the launch stream.
 *   gdn_profile_enable(1) clears previous records and starts recording;
 *   gdn_profile_enable(0) stops recording.
 *   gdn_profile_read synchronises the recorded events and reports, for the
 *   i-th distinct kernel name (0 <= i < count), its name (static string),
 *   the number of recorded launches and their summed duration in ms.
 * gdn_profile_read(i, ...) with i >= count returns GDN_ERR_SHAPE.
 */
gdn_status gdn_profile_enable(int32_t on);
gdn_status gdn_profile_count(int32_t *count);
gdn_status gdn_profile_read(int32_t index, const char **name, int64_t *launches,
                            double *total_ms);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
