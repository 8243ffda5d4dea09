/*
 * ssd.h - C ABI of the MI355X (gfx950) Mamba-2 SSD chunked-scan forward.
 *
 * The operation (per batch row r and head h):
 *
 *     H_t = a_t * H_{t-1} + x_t B_t^T,    y_t = H_t C_t + D_h x_t,
 *     a_t = exp(dt_t * A_h),  A_h = -exp(A_log_h)
 *
 * with the P x N state H carried across tokens.  The recurrence and its
 * matrix (dual) form Y = [L o (C B^T)] X are defined on "088 Mamba-2: writing
 * the recurrent state as a structured matrix" (wq-win.github.io), sections 2.1
 * and 2.2; the chunked evaluation (quadratic diagonal blocks, states passed
 * between chunks) is its section 2.3 and section 3, and key design 2 of
 * "Mamba-2 - Transformer and SSM share one algebra" (awesome.papernotes.org).
 * The decay a = exp(Delta A) is from the selective-SSM section of the "Mamba"
 * paper story (ai.tomabc.com); the skip term D x from section 2 of "Mamba and
 * state space models" (wang-x-xia.github.io); B and C shared by groups of heads
 * from key design 3 of the papernotes page.
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers to dense, contiguous, row-major
 *    arrays in the layouts given below.  The caller allocates and frees every
 *    buffer, including the workspace; the library allocates no memory.
 *  - Work is enqueued on `stream` (a hipStream_t; NULL = the default stream).
 *    No entry point synchronises the stream; errors raised by the kernels
 *    themselves surface at the caller's next synchronisation.
 *  - Every function returns SSD_OK (0) or a positive SSD_ERR_* code; nothing
 *    aborts and no C++ exception crosses the ABI.  Argument checks run on the
 *    host before any HIP call, so a rejected call has enqueued nothing.
 *  - The library keeps no per-call state; concurrent calls on different
 *    streams with disjoint outputs and workspaces are safe (except
 *    ssd_forward_noalloc, whose calls on one GPU share a static scratch array).
 *  - A call only launches kernels on `stream` (no allocation, memset, copy or
 *    synchronisation), so it may be recorded into a HIP graph by stream capture
 *    and replayed; the captured pointers must stay valid for every replay.
 */
#ifndef SSD_MI355X_H
#define SSD_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Raised when a call or a struct that was there changes; calls are added without. */
#define SSD_ABI_VERSION 5

/* Element type of x, B and C.  dt, A_log, D, init_state, y and final_state are
 * always fp32.  BF16: bf16 operands, fp32 accumulation; F32: fp32 throughout. */
typedef enum { SSD_DTYPE_F32 = 0, SSD_DTYPE_BF16 = 1 } ssd_dtype_t;

/* flags */
enum {
    /* Euler input scaling: the state is written with dt_t * x_t instead of x_t
     * (B-bar = Delta B).  D still multiplies the unscaled x_t.  Off by default:
     * the recurrence above has no Delta on x. */
    SSD_FLAG_DT_SCALES_X = 1u << 0,
    /* Step size Delta = softplus(dt + dt_bias[h]) instead of dt + dt_bias[h]
     * (the Mamba block maps its step-size projection plus a learned per-head
     * bias through softplus: the simplified Mamba block pseudocode of the
     * "Mamba" paper story).  softplus(v) = log(1 + e^v), evaluated in fp32. */
    SSD_FLAG_DT_SOFTPLUS = 1u << 1,
    /* Exact zero-order-hold input scaling: the state is written with
     * (exp(Delta A) - 1) / A * x_t, the solution over one step of
     * h' = A h + B x with x and B held constant (the pages name the
     * zero-order hold in section 2 of "Mamba and state space models" without
     * giving B-bar).  D multiplies the unscaled x_t.  Exclusive with
     * SSD_FLAG_DT_SCALES_X (both set: SSD_ERR_UNSUPPORTED). */
    SSD_FLAG_ZOH = 1u << 2
};

enum {
    SSD_OK = 0,
    SSD_ERR_NULL_POINTER = 1,   /* a required pointer is NULL                        */
    SSD_ERR_BAD_SHAPE = 2,      /* negative size, H % G != 0, nseqs inconsistent ... */
    SSD_ERR_UNSUPPORTED = 3,    /* (dtype, headdim, dstate, chunk_len) not built      */
    SSD_ERR_ALIGNMENT = 4,      /* a tensor pointer is not 16-byte aligned            */
    SSD_ERR_WORKSPACE = 5,      /* workspace NULL or smaller than ssd_workspace_size  */
    SSD_ERR_ALIAS = 6,          /* an output overlaps an input or the other output    */
    SSD_ERR_HIP = 7,            /* a HIP runtime call or kernel launch failed         */
    SSD_ERR_NO_DEVICE = 8,      /* no HIP device is available                         */
    SSD_ERR_SCRATCH = 9         /* ssd_forward_noalloc: the problem needs more scratch
                                   than SSD_NOALLOC_SCRATCH_BYTES                      */
};

/* Size of the static device scratch array of ssd_forward_noalloc (32 MiB). */
#define SSD_NOALLOC_SCRATCH_BYTES (32u << 20)

typedef struct {
    int64_t batch;      /* b: rows                                                  */
    int64_t seqlen;     /* T: tokens per row (may be 0)                             */
    int64_t nheads;     /* H                                                        */
    int64_t headdim;    /* P: channels per head (x and y)                           */
    int64_t dstate;     /* N: state size (B and C)                                  */
    int64_t ngroups;    /* G: B/C groups; head h reads group h / (H / G)            */
    int64_t chunk_len;  /* Q: chunk length of the block algorithm (see below)      */
    int64_t nseqs;      /* number of sequences: == batch without seq_idx            */
    int32_t dtype;      /* ssd_dtype_t                                              */
    uint32_t flags;     /* SSD_FLAG_*                                               */
    int32_t segments;   /* segments per row for the split-row path of ssd_forward and
                           ssd_backward: 0 lets the library choose (the default);
                           n > 0 forces n (clamped to the row's blocks), 1 no split.
                           A scheduling choice only: every value gives the same
                           function.  Must be >= 0                                  */
    int32_t reserved;   /* must be 0                                                */
} ssd_problem_t;

/* Host-only check of a problem description (no HIP call).  Supported builds:
 *   BF16: headdim in {32, 64}, dstate in {64, 128, 256}
 *   F32 : headdim in {16, 32, 64}, dstate in {16, 32, 64, 128}
 * chunk_len: 16, 32, or any positive multiple of 64.  The chunk length does
 * not change the function computed (every chunking of the sequence gives the
 * same y and final state up to rounding, section 1 of "088 Mamba-2"); the
 * kernel evaluates the sequence in blocks of 32 rows (chunk_len 16 or 32) or 64
 * rows (multiples of 64), passing the state between blocks (the past-to-future
 * parts of a diagonal block are low rank, exactly as between chunks).
 * A negative `segments` gives SSD_ERR_BAD_SHAPE, a nonzero `reserved`
 * SSD_ERR_UNSUPPORTED. */
int ssd_validate(const ssd_problem_t* p);

/* Bytes of device workspace ssd_forward needs for this problem; 0 when it needs
 * none (then workspace may be NULL) or when the problem is invalid.  A row is
 * scanned in one pass with every intermediate (C.B^T tiles, decays, the
 * carried state) on chip, unless there are at most 128 (row, head) items and
 * rows of at least 16 blocks (block: 64 tokens, or 32 for chunk_len < 64):
 * then rows are cut into segments that run in parallel, and the workspace holds
 * each segment's state (fp32 P x N) and carried decay, (batch, nheads,
 * segments - 1) of each.  The chunked algorithm's inter-chunk state passing at
 * segment granularity (section 3 of "088 Mamba-2"; key design 2 on the
 * papernotes page).  Depends on the problem only (its `segments` field forces
 * the number of segments per row); the contents need no initialisation. */
size_t ssd_workspace_size(const ssd_problem_t* p);

/* Full forward on `stream`: one kernel launch, or three when rows are split
 * into segments (see ssd_workspace_size).
 *   x          (batch, seqlen, nheads, headdim)   dtype
 *   dt         (batch, seqlen, nheads)            fp32: the step sizes, or with SSD_FLAG_DT_SOFTPLUS
 *                                                 their pre-activation (any real value)
 *   dt_bias    (nheads)                           fp32 added to dt before the step-size map, or NULL (= 0)
 *   A_log      (nheads)                           fp32; A_h = -exp(A_log[h])
 *   B, C       (batch, seqlen, ngroups, dstate)   dtype
 *   D          (nheads)                           fp32, or NULL for no skip term
 *   init_state (nseqs, nheads, headdim, dstate)   fp32, or NULL for zero initial states
 *   seq_idx    (batch, seqlen)                    int32 or NULL
 *   y          (batch, seqlen, nheads, headdim)   fp32 output
 *   final_state(nseqs, nheads, headdim, dstate)   fp32 output, or NULL
 *   workspace / workspace_bytes                   >= ssd_workspace_size(p) bytes, 256-byte aligned
 *                                                 (NULL / 0 when that size is 0)
 *
 * seq_idx packs independent sequences into rows: seq_idx[r][t] is the id of
 * the sequence token t of row r belongs to.  Ids are nondecreasing along each
 * row, global over the batch (0 .. nseqs-1), and no id appears in two rows.
 * At the first token of sequence k the state is replaced by init_state[k] (or
 * zero) and then updated by that token; final_state[k] is the state after the
 * last token of k.  No state crosses a sequence boundary.  Without seq_idx,
 * row r is sequence r (nseqs must equal batch).  Ids outside 0..nseqs-1 are
 * clamped (memory-safe, values undefined).  final_state rows of ids that never
 * occur are not written.  final_state may be the same buffer as init_state
 * (in-place state carry) only without seq_idx and when ssd_workspace_size(p)
 * is 0 (each row scanned in one piece): then every state element is read and
 * later written by the same wave.  With seq_idx, or with rows split into
 * segments that run concurrently, an in-place call is rejected with
 * SSD_ERR_ALIAS, as is any other overlap between an output and an input.
 * A row of seqlen 0 leaves its final state equal to its initial state. */
int ssd_forward(const ssd_problem_t* p,
                const void* x, const float* dt, const float* dt_bias, const float* A_log,
                const void* B, const void* C, const float* D,
                const float* init_state, const int32_t* seq_idx,
                float* y, float* final_state,
                void* workspace, size_t workspace_bytes, void* stream);

/* ssd_forward without a workspace argument, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc).  Same arguments, semantics, kernels and results as
 * ssd_forward, minus workspace / workspace_bytes: when the problem needs a
 * workspace (ssd_workspace_size(p) > 0: rows split into segments), the
 * library's own file-scope device array of SSD_NOALLOC_SCRATCH_BYTES stands in
 * for it.  A problem that needs more (ssd_workspace_size(p) >
 * ssd_noalloc_scratch_bytes()) is rejected with SSD_ERR_SCRATCH before any HIP
 * call.  The call itself allocates nothing: no hipMalloc, no hipFree, no
 * allocating library routine.  Each GPU the library runs on holds its own copy
 * of the array until the process ends; its device address is looked up once
 * per device, on the first call that needs it.  Every call on one GPU shares
 * that GPU's array, and the contents of the previous call are left in it (the
 * kernels write every scratch element they read, so nothing needs clearing):
 * calls that overlap in time on one GPU (on different streams, or from
 * different threads without ordering) race on the scratch and must not be
 * issued. */
int ssd_forward_noalloc(const ssd_problem_t* p,
                        const void* x, const float* dt, const float* dt_bias, const float* A_log,
                        const void* B, const void* C, const float* D,
                        const float* init_state, const int32_t* seq_idx,
                        float* y, float* final_state, void* stream);

/* SSD_NOALLOC_SCRATCH_BYTES, as built into the loaded library. */
size_t ssd_noalloc_scratch_bytes(void);

/* One token of the recurrence (decoding), for every row and head, on the
 * fp32 state in place:
 *     state <- a * state + x B^T,   y = state C + D x,   a = exp(dt * A_h)
 * exactly ssd_forward with seqlen 1, init_state = final_state = state (the
 * recurrence of "088 Mamba-2", section 2.1, one step at a time; a chunked
 * prefill followed by steps continues the same sequence).
 *   p          problem with seqlen == 1 and nseqs == batch (chunk_len any valid value)
 *   x          (batch, 1, nheads, headdim)   dtype
 *   dt         (batch, 1, nheads)            fp32
 *   dt_bias    (nheads) fp32, or NULL
 *   A_log      (nheads)                      fp32
 *   B, C       (batch, 1, ngroups, dstate)   dtype
 *   D          (nheads) fp32, or NULL
 *   state      (batch, nheads, headdim, dstate) fp32, read and written (required)
 *   y          (batch, 1, nheads, headdim)   fp32 output
 * The flags (Euler or zero-order-hold input scaling, softplus step size) and
 * dt_bias apply as in ssd_forward.  One kernel launch; bound by
 * reading and writing the state once.  y and state must not overlap each other
 * or any input (SSD_ERR_ALIAS). */
int ssd_step(const ssd_problem_t* p,
             const void* x, const float* dt, const float* dt_bias, const float* A_log,
             const void* B, const void* C, const float* D,
             float* state, float* y, void* stream);

/* Bytes of device workspace ssd_backward needs (0 if the problem is invalid):
 * per-token scalars and dt transposed to (batch, nheads, seqlen), per-(sequence,
 * head) scalars, a table of the packed sequences, and, when a group holds more than one
 * head, each head's dB and dC contribution, (batch, seqlen, nheads, dstate)
 * each in the input type (bf16 or fp32), before the fp32 sum over the group;
 * and each 64-token (bf16) or 32-token (fp32) block's incoming state,
 * (batch, nheads, blocks, headdim, dstate) in the input type.  The contents need no
 * initialisation. */
size_t ssd_backward_workspace_size(const ssd_problem_t* p);

/* Gradients of the forward map (training).  For a scalar loss L with
 * dL/dy = dy and dL/dfinal_state = dfinal (NULL: L does not depend on the
 * final states), writes dL/d(every input).  The pages give no backward
 * algorithm: this is the chain rule applied to the recurrence of "088
 * Mamba-2" (section 2.1), G_t = dL/dS_t = dy_t C_t^T + a_{t+1} G_{t+1},
 * evaluated with the same block (dual) form as the forward (sections 2.2-3).
 *   inputs     as ssd_forward (same problem, flags and tensors), plus
 *   dy         (batch, seqlen, nheads, headdim)   fp32
 *   dfinal     (nseqs, nheads, headdim, dstate)   fp32, or NULL
 *   outputs (fp32):
 *   dx         (batch, seqlen, nheads, headdim)
 *   ddt        (batch, seqlen, nheads)     with respect to the dt input (through softplus if flagged)
 *   dA_log     (nheads)
 *   dB, dC     (batch, seqlen, ngroups, dstate)   summed over the heads of each group
 *   dD         (nheads), or NULL
 *   dinit      (nseqs, nheads, headdim, dstate), or NULL (the gradient with respect to
 *              init_state, also when init_state is NULL, i.e. at a zero initial state)
 *   ddt_bias   (nheads), or NULL
 *   workspace  >= ssd_backward_workspace_size(p) bytes, 256-byte aligned
 * With seq_idx (packed sequences, as in ssd_forward) dfinal and dinit are per
 * sequence; a sequence id that does not occur gets dinit = 0.  Each (sequence,
 * head) is walked on its own, in blocks aligned to the sequence's first token;
 * a device-side table of the sequences is built from seq_idx first (the host
 * never reads it).  Supported shapes: BF16 headdim 32 or 64 with dstate 64,
 * 128 or 256; F32 headdim 16, 32 or 64 with dstate 16 .. 128.  Outputs must not
 * overlap any input, the workspace or each other (SSD_ERR_ALIAS).  x, B, C, dy,
 * dx, dB, dC, init_state, dfinal and dinit need 16-byte alignment, the rest 4.
 * Two kernel launches walk each (row, head) once forwards and once backwards
 * with the state on chip; then, with more than one head per group, a sum of the
 * heads' dB and dC; then the per-head sums over rows.  Per-head sums are taken in
 * a fixed order, so results are deterministic. */
int ssd_backward(const ssd_problem_t* p,
                 const void* x, const float* dt, const float* dt_bias, const float* A_log,
                 const void* B, const void* C, const float* D,
                 const float* init_state, const int32_t* seq_idx,
                 const float* dy, const float* dfinal,
                 float* dx, float* ddt, float* dA_log, float* dB, float* dC,
                 float* dD, float* dinit, float* ddt_bias,
                 void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------
 * The operators around the scan in a Mamba layer.  The conventions at the top of
 * this file hold for them too, with three differences: a tensor argument needs only
 * the alignment of its element type; the inputs named with an `ld` field may be
 * slices of wider rows (an `ld` is the distance in elements from one token to the
 * next, over the whole batch, channels being contiguous); and every parameter,
 * state and gradient is fp32 whatever the type of the activations.
 * ------------------------------------------------------------------------------ */

/* conv flags */
enum {
    SSD_CONV_SILU = 1u << 0    /* y = silu(pre) instead of pre */
};

typedef struct {
    int64_t batch;      /* rows                                                     */
    int64_t seqlen;     /* tokens per row (may be 0)                                */
    int64_t channels;   /* D                                                        */
    int64_t nseqs;      /* number of sequences: == batch without seq_idx            */
    int64_t ldx;        /* elements from one token of x to the next, >= channels, < 2^31 */
    int32_t width;      /* K: taps, 2 to 4                                          */
    int32_t dtype;      /* ssd_dtype_t of x and y                                   */
    uint32_t flags;     /* SSD_CONV_*                                               */
    int32_t reserved;   /* must be 0                                                */
} ssd_conv_problem_t;

/* The short causal convolution over each channel (the conv layer before the scan in
 * the Mamba block; simplified block pseudocode of the "Mamba" paper story):
 *     pre[t][d] = bias[d] + sum_{j=0}^{K-1} weight[d][K-1-j] in[t-j][d],
 *     y = pre, or silu(pre) = pre / (1 + exp(-pre)).
 * in[t-j] is the token j back in the same sequence; before the sequence's first token
 * it is the matching row of its initial state (K-1 rows, oldest first), or zero.
 *   x           (batch, seqlen, channels)      dtype, tokens ldx apart
 *   weight      (channels, width)              fp32
 *   bias        (channels)                     fp32, or NULL
 *   init_state  (nseqs, width-1, channels)     fp32, or NULL for zeros
 *   seq_idx     (batch, seqlen)                int32 or NULL, as in ssd_forward
 *   y           (batch, seqlen, channels)      dtype, output
 *   final_state (nseqs, width-1, channels)     fp32 output or NULL: each sequence's last
 *               K-1 inputs, of a shorter sequence those of its initial state before them.
 *               Rows of ids that do not occur are not written.
 * Outputs must not overlap inputs or each other (SSD_ERR_ALIAS): the tokens of a row are
 * spread over workgroups, so the state is not carried in place.  One kernel launch. */
int ssd_conv_forward(const ssd_conv_problem_t* p, const void* x, const float* weight, const float* bias,
                     const float* init_state, const int32_t* seq_idx, void* y, float* final_state, void* stream);

/* Bytes of device workspace ssd_conv_backward needs (0 for an invalid problem): partial
 * sums of the weight and bias gradients. */
size_t ssd_conv_backward_workspace_size(const ssd_conv_problem_t* p);

/* Gradients of L for dL/dy = dy (fp32) and dL/dfinal_state = dfinal (fp32, or NULL), all
 * fp32 and dense: dx (batch, seqlen, channels), dweight (channels, width), dbias
 * (channels) or NULL, dinit (nseqs, width-1, channels) or NULL (at a zero state when
 * init_state is NULL; zero for ids that do not occur).  workspace: 256-byte aligned.
 * The sums over tokens have a fixed order: results are deterministic. */
int ssd_conv_backward(const ssd_conv_problem_t* p, const void* x, const float* weight, const float* bias,
                      const float* init_state, const int32_t* seq_idx, const float* dy, const float* dfinal,
                      float* dx, float* dweight, float* dbias, float* dinit, void* workspace, size_t workspace_bytes,
                      void* stream);

/* One token (decoding): ssd_conv_forward with seqlen 1 and nseqs == batch, from `state` to
 * `state_out`, which may be the same buffer (in place) or one that does not overlap it. */
int ssd_conv_step(const ssd_conv_problem_t* p, const void* x, const float* weight, const float* bias,
                  const float* state, float* state_out, void* y, void* stream);

typedef struct {
    int64_t batch;      /* rows                                                     */
    int64_t seqlen;     /* tokens per row (may be 0)                                */
    int64_t channels;   /* D, < 2^25                                                */
    int64_t dstate;     /* N: 8, 16, 32 or 64                                       */
    int64_t ngroups;    /* G: B/C groups; channel d reads group d / (D / G)         */
    int64_t nseqs;      /* number of sequences: == batch without seq_idx            */
    int64_t ldx, lddt, ldz;   /* elements from one token to the next, >= channels, < 2^25
                                 (ssd_selective_step: < 2^31)                       */
    int64_t ldb, ldc;   /* the same of B and C, >= ngroups * dstate                 */
    int32_t dtype;      /* ssd_dtype_t of x, dt, B, C, z and y                      */
    uint32_t flags;     /* SSD_FLAG_DT_SOFTPLUS or 0                                */
    int32_t segments;   /* segments per row, as in ssd_problem_t: 0 lets the library choose */
    int32_t reserved;   /* must be 0                                                */
} ssd_selective_problem_t;

/* The selective scan with a decay per channel and state (the scan of the Mamba-1 block;
 * selective-SSM section of the "Mamba" paper story):
 *     h_t[d][n] = exp(step_t[d] A[d][n]) h_{t-1}[d][n] + step_t[d] x_t[d] B_t[n],
 *     y_t[d] = sum_n C_t[n] h_t[d][n] + D[d] x_t[d],   times silu(z_t[d]) with z,
 * A = -exp(A_log), step = dt + dt_bias, through softplus with SSD_FLAG_DT_SOFTPLUS.
 *   x, dt       (batch, seqlen, channels)          dtype; tokens ldx, lddt apart
 *   dt_bias     (channels)                         fp32, or NULL (= 0)
 *   A_log       (channels, dstate)                 fp32
 *   B, C        (batch, seqlen, ngroups, dstate)   dtype; tokens ldb, ldc apart
 *   D           (channels)                         fp32, or NULL for no skip term
 *   z           (batch, seqlen, channels)          dtype, tokens ldz apart, or NULL for no gate
 *   init_state  (nseqs, channels, dstate)          fp32, or NULL for zeros
 *   seq_idx     (batch, seqlen)                    int32 or NULL, as in ssd_forward
 *   y           (batch, seqlen, channels)          dtype, output
 *   final_state (nseqs, channels, dstate)          fp32 output, or NULL; rows of ids that do
 *                                                  not occur are not written
 *   workspace   >= ssd_selective_workspace_size(p) bytes, 256-byte aligned (NULL / 0 when 0)
 * The recurrence runs in fp32.  Rows are cut into segments (one launch becomes three) when
 * there are too few channels and rows to fill the chip.  Step sizes are meant to be >= 0, so
 * that states decay; with negative ones they grow, and in a cut row the growth exp(A sum of
 * steps) of a whole segment has to be finite in fp32, also where the state is zero.  Outputs must not overlap inputs,
 * the workspace or each other (SSD_ERR_ALIAS); the state is not carried in place. */
size_t ssd_selective_workspace_size(const ssd_selective_problem_t* p);
int ssd_selective_forward(const ssd_selective_problem_t* p, const void* x, const void* dt, const float* dt_bias,
                          const float* A_log, const void* B, const void* C, const float* D, const void* z,
                          const float* init_state, const int32_t* seq_idx, void* y, float* final_state, void* workspace,
                          size_t workspace_bytes, void* stream);

/* One token (decoding): ssd_selective_forward with seqlen 1 and nseqs == batch, from `state`
 * to `state_out`, which may be the same buffer (in place) or one that does not overlap it.
 * One launch, bound by reading and writing the state. */
int ssd_selective_step(const ssd_selective_problem_t* p, const void* x, const void* dt, const float* dt_bias,
                       const float* A_log, const void* B, const void* C, const float* D, const void* z,
                       const float* state, float* state_out, void* y, void* stream);

/* Gradients of L for dL/dy = dy (fp32) and dL/dfinal_state = dfinal (fp32, or NULL), all
 * fp32 and dense, shaped like their inputs: dx, ddt (through softplus if flagged), dA_log,
 * dB, dC (summed over the channels of a group), dz (required with z), and, each NULL if not
 * wanted, dD, dinit (at a zero state when init_state is NULL; zero for ids that do not
 * occur) and ddt_bias.  workspace: >= ssd_selective_backward_workspace_size(p) bytes,
 * 256-byte aligned: a state every eight tokens, and the channel blocks' parts of dB and dC.
 * Sums are taken in a fixed order: results are deterministic.  Negative step sizes: as in
 * ssd_selective_forward. */
size_t ssd_selective_backward_workspace_size(const ssd_selective_problem_t* p);
int ssd_selective_backward(const ssd_selective_problem_t* p, const void* x, const void* dt, const float* dt_bias,
                           const float* A_log, const void* B, const void* C, const float* D, const void* z,
                           const float* init_state, const int32_t* seq_idx, const float* dy, const float* dfinal,
                           float* dx, float* ddt, float* dA_log, float* dB, float* dC, float* dD, float* dz,
                           float* dinit, float* ddt_bias, void* workspace, size_t workspace_bytes, void* stream);

/* norm flags */
enum {
    SSD_NORM_GATE_FIRST = 1u << 0    /* gate before the norm (else after it) */
};

typedef struct {
    int64_t rows;
    int64_t channels;     /* D                                                              */
    int64_t group_size;   /* consecutive channels normed together; divides channels; <= 32768 */
    int64_t ldx;          /* elements from one row of x to the next, >= channels, < 2^31    */
    int64_t ldz;          /* the same of z, or of residual                                  */
    float eps;            /* >= 0                                                           */
    int32_t x_dtype;      /* ssd_dtype_t of x                                               */
    int32_t dtype;        /* ssd_dtype_t of z and out                                       */
    uint32_t flags;       /* SSD_NORM_*                                                     */
    int32_t reserved;     /* must be 0                                                      */
} ssd_norm_problem_t;

/* The root-mean-square norm after the scan with its gate, per row and group of channels
 * (the gate beside the scan in the Mamba block's simplified pseudocode, "Mamba" paper
 * story; the norm after it, which the pages do not detail, read as
 * v / sqrt(mean(v^2) + eps)):
 *     gate first: u = x silu(z), out = u / sqrt(mean(u^2) + eps) weight
 *     gate after: out = x / sqrt(mean(x^2) + eps) weight silu(z)
 *   x      (rows, channels)   x_dtype: fp32 (the scan's y) or dtype; rows ldx apart
 *   z      (rows, channels)   dtype; rows ldz apart
 *   weight (channels)         fp32
 *   out    (rows, channels)   dtype, output; overlaps no input (SSD_ERR_ALIAS) */
int ssd_gated_norm_forward(const ssd_norm_problem_t* p, const void* x, const void* z, const float* weight, void* out,
                           void* stream);

/* Gradients for dL/dout = dout (fp32): dx, dz (rows, channels) and dweight (channels), fp32
 * and dense.  workspace: 256-byte aligned, of the size given (0 for an invalid problem). */
size_t ssd_gated_norm_backward_workspace_size(const ssd_norm_problem_t* p);
int ssd_gated_norm_backward(const ssd_norm_problem_t* p, const void* x, const void* z, const float* weight,
                            const float* dout, float* dx, float* dz, float* dweight, void* workspace,
                            size_t workspace_bytes, void* stream);

/* The norm before a block with its residual addition:
 *     residual_out = residual + scale x,  out = residual_out / sqrt(mean(residual_out^2) + eps) weight
 * over whole rows (group_size == channels, x_dtype == dtype, flags 0).
 *   x            (rows, channels)   dtype, rows ldx apart: the previous block's output
 *   residual     (rows, channels)   fp32, rows ldz apart, or NULL (the stream starts here)
 *   weight       (channels)         fp32
 *   scale        (channels)         fp32, or NULL for 1
 *   out          (rows, channels)   dtype, output
 *   residual_out (rows, channels)   fp32, output; may be `residual` itself when that is
 *                dense (in place).  Any other overlap is SSD_ERR_ALIAS. */
int ssd_residual_norm_forward(const ssd_norm_problem_t* p, const void* x, const float* residual, const float* weight,
                              const float* scale, void* out, float* residual_out, void* stream);

/* Gradients for dL/dout = dout and dL/dresidual_out = dresidual_out (NULL: nothing else
 * uses the stream), from the residual_out that the forward wrote.  dresidual (rows,
 * channels) is also the gradient of x when scale is NULL; with a scale, dx = scale
 * dresidual and dscale (channels) are written and x is read (without one, x, dx and
 * dscale may be NULL).  dweight (channels).  All fp32 and dense.  `scaled`: whether a
 * scale will be given. */
size_t ssd_residual_norm_backward_workspace_size(const ssd_norm_problem_t* p, int scaled);
int ssd_residual_norm_backward(const ssd_norm_problem_t* p, const void* x, const float* residual_out,
                               const float* weight, const float* scale, const float* dout, const float* dresidual_out,
                               float* dx, float* dresidual, float* dweight, float* dscale, void* workspace,
                               size_t workspace_bytes, void* stream);

typedef struct {
    int64_t batch;      /* rows                                                     */
    int64_t seqlen;     /* tokens per row (may be 0)                                */
    int64_t channels;   /* D                                                        */
    int64_t nseqs;      /* number of sequences: == batch without seq_idx            */
    int64_t ldx, ldr, ldi, ldz;   /* elements from one token to the next, >= channels, < 2^31 */
    int32_t dtype;      /* ssd_dtype_t of x, r, i, z and y                          */
    uint32_t flags;     /* must be 0                                                */
} ssd_recurrence_problem_t;

/* The gated linear recurrence: one state per channel, its decay and the scale of its input
 * from gates of the same token (sigma(v) = 1 / (1 + e^-v)):
 *     a_t = exp(A[d] sigma(r_t)),    A = -exp(A_log),
 *     h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigma(i_t) x_t,
 *     y_t = h_t,   times silu(z_t) with z.
 *   x, r, i     (batch, seqlen, channels)   dtype; tokens ldx, ldr, ldi apart
 *   A_log       (channels)                  fp32
 *   z           (batch, seqlen, channels)   dtype, tokens ldz apart, or NULL for no gate
 *   init_state  (nseqs, channels)           fp32, or NULL for zeros
 *   seq_idx     (batch, seqlen)             int32 or NULL, as in ssd_forward
 *   y           (batch, seqlen, channels)   dtype, output
 *   final_state (nseqs, channels)           fp32 output, or NULL; rows of ids that do not occur
 *                                           are not written
 *   workspace   >= ssd_recurrence_workspace_size(p) bytes, 256-byte aligned (NULL / 0 when 0)
 * The recurrence runs in fp32; 1 - a and 1 - a^2 are formed without cancellation, a small a keeps
 * its own relative precision.  A_log counts as at most 88, sigma or A sigma(r) below 2^-126 as 0.
 * An infinite input or state makes its channel Inf or NaN from its token to the end of its
 * sequence; nothing crosses into another sequence.  Rows of more tokens than a workgroup holds
 * (where the workspace size is not 0: over 256 tokens in bf16, over 128 in fp32 and in rows of fewer
 * than eight channels) take two launches, the first of which zeroes the workspace: it holds what
 * workgroups of this call tell each other, so two calls that run at the same time need one each (in
 * one workspace both still end, but their outputs are undefined: NaN, values of neither, or not
 * written).  Outputs must not overlap inputs, the workspace or each other (SSD_ERR_ALIAS); the state
 * is not carried in place. */
size_t ssd_recurrence_workspace_size(const ssd_recurrence_problem_t* p);
int ssd_recurrence_forward(const ssd_recurrence_problem_t* p, const void* x, const void* r, const void* i,
                           const float* A_log, const void* z, const float* init_state, const int32_t* seq_idx, void* y,
                           float* final_state, void* workspace, size_t workspace_bytes, void* stream);

/* One token (decoding): ssd_recurrence_forward with seqlen 1 and nseqs == batch, from `state`
 * to `state_out`, which may be the same buffer (in place) or one that does not overlap it. */
int ssd_recurrence_step(const ssd_recurrence_problem_t* p, const void* x, const void* r, const void* i,
                        const float* A_log, const void* z, const float* state, float* state_out, void* y, void* stream);

/* Gradients of L for dL/dy = dy (fp32) and dL/dfinal_state = dfinal (fp32, or NULL), all fp32
 * and dense, shaped like their inputs: dx, dr, di, dA_log, dz (required with z) and dinit (NULL
 * if not wanted; at a zero state when init_state is NULL, zero for ids that do not occur).
 * workspace: >= ssd_recurrence_backward_workspace_size(p) bytes, 256-byte aligned.  Sums are
 * taken in a fixed order: results are deterministic. */
size_t ssd_recurrence_backward_workspace_size(const ssd_recurrence_problem_t* p);
int ssd_recurrence_backward(const ssd_recurrence_problem_t* p, const void* x, const void* r, const void* i,
                            const float* A_log, const void* z, const float* init_state, const int32_t* seq_idx,
                            const float* dy, const float* dfinal, float* dx, float* dr, float* di, float* dA_log,
                            float* dz, float* dinit, void* workspace, size_t workspace_bytes, void* stream);

/* rotary flags */
enum {
    SSD_ROTARY_INTERLEAVED = 1u << 0    /* pairs are channels 2j, 2j + 1 (else j, j + rotary_dim / 2) */
};

typedef struct {
    int64_t tokens;       /* over the whole batch                                            */
    int64_t seqlen;       /* without positions, token t has position t % seqlen; >= 1, <= 2^31 */
    int64_t b_heads;      /* heads (groups) of B: keys                                       */
    int64_t c_heads;      /* heads (groups) of C: queries                                    */
    int64_t headdim;      /* N: channels of a head, <= 1024                                  */
    int64_t rotary_dim;   /* channels rotated, from the first on: even, 0 to headdim         */
    int64_t ldb, ldc;     /* elements from one token to the next, >= heads * headdim, < 2^31 */
    float eps;            /* >= 0                                                            */
    int32_t dtype;        /* ssd_dtype_t of B, C and the outputs                             */
    uint32_t flags;       /* SSD_ROTARY_*                                                    */
    int32_t reserved;     /* must be 0                                                       */
} ssd_rotary_problem_t;

/* The root-mean-square norm of B and C per head with the rotation by position, in one pass
 * (C plays the query, B the key of the dual form, so rotating both by their tokens' positions
 * makes the scan see C_t R(t - s) B_s, a decay with a complex factor):
 *     v = u / sqrt(mean(u^2) + eps) weight        per token and head,
 *     (out_p, out_q) = (v_p cos w - v_q sin w, v_p sin w + v_q cos w),   w = position freqs[j],
 * for the pairs (p, q) of the first rotary_dim channels, pair j; the rest of v passes as it is.
 * The angle is taken in fp64, so positions may be any int32.
 *   B, C       (tokens, heads, headdim)   dtype; tokens ldb, ldc apart, heads dense
 *   b_weight, c_weight  (headdim)         fp32, shared by the heads
 *   freqs      (rotary_dim / 2)           fp32: angle per position (NULL when rotary_dim is 0)
 *   positions  (tokens)                   int32, or NULL: t % seqlen
 *   B_out, C_out  (tokens, heads, headdim)  dtype, dense outputs, as ssd_forward takes them
 * Outputs must not overlap inputs or each other (SSD_ERR_ALIAS).  One kernel launch. */
int ssd_rotary_norm_forward(const ssd_rotary_problem_t* p, const void* B, const void* C, const float* b_weight,
                            const float* c_weight, const float* freqs, const int32_t* positions, void* B_out,
                            void* C_out, void* stream);

/* Gradients for dL/dB_out = dB_out and dL/dC_out = dC_out (fp32, dense): dB, dC (tokens, heads,
 * headdim), db_weight and dc_weight (headdim), fp32 and dense; freqs are constants.
 * workspace: 256-byte aligned, of the size given (0 for an invalid problem).  Sums are taken in
 * a fixed order: results are deterministic. */
size_t ssd_rotary_norm_backward_workspace_size(const ssd_rotary_problem_t* p);
int ssd_rotary_norm_backward(const ssd_rotary_problem_t* p, const void* B, const void* C, const float* b_weight,
                             const float* c_weight, const float* freqs, const int32_t* positions, const float* dB_out,
                             const float* dC_out, float* dB, float* dC, float* db_weight, float* dc_weight,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Static description of an error code. */
const char* ssd_strerror(int status);

/* SSD_ABI_VERSION of the loaded library. */
int ssd_version(void);

#ifdef __cplusplus
}
#endif
#endif /* SSD_MI355X_H */
